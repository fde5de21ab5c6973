"""Plain 64-bit forms of the paged operators (test helpers; numpy and the oracle only).

Tolerances of the paged attention. Every rounding is at most half a step (fp16 2^-11
relative) and on average over a row's elements about 2^-11 / sqrt(3) = 2.8e-4. The output
passes: the un-rotation matrix (one rounding per entry), the accumulated o (one), the
weights P and P times the V scale (two, or one for the weight and one for c * scale), and
the final rounding: sqrt(5) * 2.8e-4 = 6.3e-4 of the row's norm. The scores pass the query
matrix and the rotated query (and c * scale in the prompt kernel): an error of at most
sqrt(3) * 2.8e-4 of |q~| |k~| / sqrt(D) * sigma_rms, which with |score| up to about 3 is an
absolute 1.5e-3 per score and the same relative change of a weight; independent over
tokens, it moves the output by at most 1.5e-3 of the weighted spread of V, itself of the
output's size where few tokens dominate. Together below 2e-3, the suite's rule for a row;
where scores reach S the middle term grows with S / 3.
"""
import numpy as np

import oracle


def plan_step(kv, q, table, free, head, P, n_slots):
    """kvq_page_plan by a loop over the requests. Returns a dict of what it writes."""
    kv, q = [max(int(x), 0) for x in kv], [max(int(x), 0) for x in q]
    table = np.array(table, copy=True)
    head = min(max(int(head), 0), len(free))
    room, upto, got, refused, total = len(free) - head, 0, 0, 0, 0
    slots, pos, starts, kv_out = [], [], [0], []
    for b, (a, n) in enumerate(zip(kv, q)):
        have, want = -(-a // P), -(-(a + n) // P)
        fits = want <= table.shape[1]
        need = want - have if fits else 0
        first = upto
        upto += need
        served = fits and (need == 0 or upto <= room)
        if served:
            table[b, have:want] = free[head + first:head + first + need]
            got += need
        else:
            refused += 1
        for j in range(n):
            t = a + j
            pos.append(t)
            slots.append(table[b, t // P] * P + t % P if served else -1)
        starts.append(starts[-1] + n)
        kv_out.append(a + n if served else a)
    total = len(slots)
    pad = max(0, n_slots - total)
    return dict(slots=np.array((slots + [-1] * pad)[:n_slots], np.int32),
                positions=np.array((pos + [-1] * pad)[:n_slots], np.int32), q_starts=np.array(starts, np.int32),
                kv_lens=np.array(kv_out, np.int32), table=table, head=head + got,
                info=np.array([total, got, refused, upto], np.int32))


def rows_at(pages, slots, P):
    """[n, Hkv, .] rows of pages [num_pages, Hkv, P, .] at slots."""
    slots = np.asarray(slots)
    return pages[slots // P, :, slots % P]


def decoded(codes, scales, slots, P, params, G, xf, bits):
    """x_hat fp64 [n, Hkv, D] of the rows at slots."""
    return oracle.decode(rows_at(codes, slots, P), rows_at(scales, slots, P), *params, G, xf, bits)


def attend(q, kc, ks, vc, vs, table, kv_lens, q_lens, kp, vp, G, xf, bits, window=0, sigma=None):
    """Causal attention, fp64 [sum(q_lens), Hq, D]; only attended rows of the pages are touched."""
    P, Hkv = kc.shape[2], kc.shape[1]
    n, Hq, D = q.shape
    out = np.zeros((n, Hq, D))
    sigma = 1.0 / np.sqrt(D) if sigma is None else sigma
    at = 0
    for b, (L, m) in enumerate(zip(kv_lens, q_lens)):
        first = max(0, L - m + 1 - window) if window else 0
        t = np.arange(first, L)
        if m and len(t):
            slots = np.asarray(table[b]).astype(np.int64)[t // P] * P + t % P
            with np.errstate(invalid="ignore", over="ignore"):
                K, V = decoded(kc, ks, slots, P, kp, G, xf, bits), decoded(vc, vs, slots, P, vp, G, xf, bits)
            for j in range(m):
                p = L - m + j
                use = (t <= p) & ((t > p - window) if window else True)
                if not use.any():
                    continue
                for h in range(Hq):
                    z = K[use, h // (Hq // Hkv)] @ q[at + j, h].astype(np.float64) * sigma
                    w = np.exp(z - z.max())
                    out[at + j, h] = w @ V[use, h // (Hq // Hkv)] / w.sum()
        at += m
    return out
