"""The operators of the paged 4-bit (and 8-bit) KV cache, as cases to be measured and compared.

Four operators, each in its plain form (elementary torch operations) and as the library's call:

  plan    block tables and slot maps of one serving step, built on the GPU from request lengths
  store   rows of K and V encoded into cache pages at given slots, then read back
  fetch   cached rows at given slots decoded to fp16
  attend  attention of ragged queries over the pages (one token per request, or several, causal)

A cached vector x (fp16, head_dim D) is held as codes c and fp16 group scales of
y = lambda * (Q (s * x)): s fixed signs, Q the orthonormal real DFT (rows DC, cos 1, sin 1, ...,
Nyquist) or the normalised Hadamard matrix, lambda a factor per channel; per group of G channels
scale = fp16(min(absmax / Qmax, 65504)), c = clamp(round(y / scale), -Qmax, Qmax), Qmax 7 (4 bits)
or 127 (8 bits). Pages: codes u8 [pages, kv heads, page size, D * bits / 8] (4 bits: channel 2j in
the low half of byte j), scales fp16 [pages, kv heads, page size, D / G]. Slot = page * page size +
place in the page.
"""
import math
import random

import torch

own = False

DEV = "cuda"

# The head geometries are the ones the benchmark and the tests use: 12 query / 2 KV heads of 128,
# 32 / 8 of 128, 64 / 8 of 128 and 4 / 1 of 256.
GEOMETRIES = [(12, 2, 128), (32, 8, 128), (64, 8, 128), (4, 1, 256)]


# --------------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of 32 requests: each gets one token; the smallest call, latency alone
        dict(name="plan-step", op="plan", B=32, fresh=0.0, q_hi=1, kv_hi=4096, page=16, tight=False, mix=1),
        # a large serving step: decode rows mixed with prompts up to 1024 tokens, the free list too
        # short for the last of them
        dict(name="plan-mixed", op="plan", B=2048, fresh=0.2, q_hi=1024, kv_hi=8192, page=64, tight=True, mix=2),
        # the new token of 32 requests written to the cache and read back
        dict(name="store-step", op="store", n=32, Hkv=8, D=128, G=32, bits=4, xf="srft", page=16, pad=0, mix=3),
        # a prompt batch of 16K tokens written to the cache, with padded rows behind it, and read back
        dict(name="store-prompt", op="store", n=16384, Hkv=8, D=128, G=32, bits=4, xf="srft", page=64, pad=77, mix=4),
        # an odd prompt with 256-wide heads and 8-bit Hadamard codes
        dict(name="store-wide8", op="store", n=5003, Hkv=1, D=256, G=16, bits=8, xf="srht", page=32, pad=5, mix=5),
        # a cached prefix of 32K tokens brought back to fp16
        dict(name="fetch-prefix", op="fetch", n=32768, Hkv=8, D=128, G=32, bits=4, xf="srft", page=64, pad=0, mix=6),
        # a short odd piece of a cache with 256-wide heads
        dict(name="fetch-odd", op="fetch", n=999, Hkv=1, D=256, G=32, bits=4, xf="srft", page=16, pad=3, mix=7),
        # one request, one token, a short cache: the least latency a layer can have
        dict(name="attend-one", op="attend", B=1, Hq=12, Hkv=2, D=128, G=32, bits=4, xf="srft", page=16, q_hi=1,
             kv_lo=700, kv_hi=700, window=0, mix=8),
        # a decode batch of ragged lengths
        dict(name="attend-batch", op="attend", B=64, Hq=32, Hkv=8, D=128, G=32, bits=4, xf="srft", page=16, q_hi=1,
             kv_lo=200, kv_hi=8192, window=0, mix=9),
        # few requests with very long caches
        dict(name="attend-long", op="attend", B=4, Hq=64, Hkv=8, D=128, G=32, bits=4, xf="srft", page=64, q_hi=1,
             kv_lo=90000, kv_hi=131072, window=0, mix=10),
        # several tokens per request checked at once (drafted tokens), 256-wide heads, sliding window
        dict(name="attend-draft", op="attend", B=8, Hq=4, Hkv=1, D=256, G=32, bits=4, xf="srft", page=32, q_hi=6,
             kv_lo=1000, kv_hi=16384, window=1024, mix=11),
        # prompts worked off in chunks of up to 2048 tokens on caches up to 16K tokens
        dict(name="attend-chunk", op="attend", B=2, Hq=32, Hkv=8, D=128, G=32, bits=4, xf="srft", page=64, q_hi=2048,
             kv_lo=8192, kv_hi=16384, window=0, mix=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "store", "fetch", "attend", "attend", "attend"])
    mix = rng.randrange(1 << 20)
    if op == "plan":
        return dict(op=op, B=_log(rng, 1, 2048), fresh=rng.choice([0.0, 0.1, 0.2]), q_hi=_log(rng, 1, 1024),
                    kv_hi=_log(rng, 16, 8192), page=rng.choice([16, 32, 64, 128]), tight=rng.random() < 0.3, mix=mix)
    Hq, Hkv, D = rng.choice(GEOMETRIES)
    form = dict(D=D, G=rng.choice([32, 32, 16]), bits=rng.choice([4, 4, 8]), xf=rng.choice(["srft", "srft", "srht"]),
                page=rng.choice([16, 32, 64, 128]), mix=mix)
    if op == "store" or op == "fetch":
        return dict(op=op, n=_log(rng, 1, 16384 if op == "store" else 32768), Hkv=Hkv, pad=rng.choice([0, 0, 1, 9]), **form)
    kind = rng.choice(["step", "step", "few", "chunk"])
    if kind == "step":     # one token per request: requests x cached tokens up to 256K
        B = _log(rng, 1, 64)
        q_hi, kv_hi = 1, _log(rng, 1, min(131072, 262144 // B))
    elif kind == "few":    # a handful of tokens per request
        B = _log(rng, 1, 32)
        q_hi, kv_hi = rng.randint(2, 9), _log(rng, 16, 65536 // B)
    else:                  # prompt chunks
        B = rng.randint(1, 3)
        q_hi = _log(rng, 10, 2048)
        # query rows x cached tokens at most what the largest listed chunk has
        kv_hi = _log(rng, q_hi, max(q_hi, min(16384, (1 << 37) // (B * q_hi * Hq * D))))
    window = _log(rng, 16, kv_hi + 16) if rng.random() < 0.3 else 0
    return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, q_hi=q_hi, kv_lo=max(1, kv_hi // rng.choice([1, 4, 32])), kv_hi=kv_hi,
                window=window, **form)


def _lens(case):
    """The step's request lengths (host lists): cached tokens before it and new tokens, from the case alone."""
    r = random.Random(case["mix"])
    if case["op"] == "plan":
        kv, q = [], []
        for _ in range(case["B"]):
            if r.random() < case["fresh"]:          # a new prompt
                kv.append(0)
                q.append(r.randint(1, case["q_hi"]))
            else:                                   # a running request; now and then an idle row
                kv.append(_log(r, 1, case["kv_hi"]))
                q.append(0 if r.random() < 0.03 else 1)
        return kv, q
    # attention: lengths after the step's tokens were stored
    q = [case["q_hi"] if i == 0 else r.randint(max(1, case["q_hi"] // 2), case["q_hi"]) for i in range(case["B"])]
    kv = [max(n, case["kv_hi"] if i == 0 else _log(r, case["kv_lo"], case["kv_hi"])) for i, n in enumerate(q)]
    return kv, q


def work(case):
    if case["op"] == "plan":
        kv, q = _lens(case)
        P = case["page"]
        new = sum(-(-(a + b) // P) - -(-a // P) for a, b in zip(kv, q))
        # lengths in; starts and lengths out; slot and position of each token; free-list entry and table entry per page
        return {"bytes": 4.0 * (4 * len(kv) + 2 * sum(q) + 2 * new), "flops": 0.0}
    D, G, bits, Hkv = case["D"], case["G"], case["bits"], case["Hkv"]
    row = D * bits / 8 + 2 * D / G
    dense = 2.0 * D * D                             # one vector through the rotation as a product
    if case["op"] == "store":
        vec = 2.0 * case["n"] * Hkv                 # K and V
        # fp16 in, packed out, packed in, fp16 out, a slot per token
        return {"bytes": vec * (4 * D + 2 * row) + 4.0 * case["n"], "flops": 2 * vec * dense}
    if case["op"] == "fetch":
        vec = case["n"] * float(Hkv)
        return {"bytes": vec * (2 * D + row) + 4.0 * case["n"], "flops": vec * dense}
    kv, q = _lens(case)
    W, tokens, pairs = case["window"], 0, 0
    for L, n in zip(kv, q):
        first = max(0, L - n + 1 - W) if W else 0
        tokens += L - first
        if not W:
            pairs += n * L - n * (n - 1) // 2
        else:
            pairs += sum(min(W, p + 1) for p in range(L - n, L))
    N = sum(q)
    return {"bytes": 2.0 * tokens * Hkv * row + 4.0 * N * case["Hq"] * D,
            "flops": 4.0 * pairs * case["Hq"] * D}


# --------------------------------------------------------------------------- inputs
def _basis(D, xf, device):
    """The orthonormal rotation Q, row = channel."""
    n = torch.arange(D, device=device)
    if xf == "srht":
        m = n[:, None] & n[None, :]
        par = torch.zeros_like(m)
        for b in range(D.bit_length()):
            par = par ^ ((m >> b) & 1)
        return (1 - 2 * par).to(torch.float64) / math.sqrt(D)
    k = (n + 1) // 2
    ang = (2.0 * math.pi / D) * ((k[:, None] * n[None, :]) % D).to(torch.float64)
    Q = math.sqrt(2.0 / D) * torch.where((n % 2 == 1)[:, None], torch.cos(ang), torch.sin(ang))
    Q[0] = 1.0 / math.sqrt(D)
    Q[D - 1] = (1.0 - 2.0 * (n % 2)).to(torch.float64) / math.sqrt(D)
    return Q


def _packed(g, pages, case, spread):
    """Pages as a cache holds them: groups of normal values, quantised; `spread` is the values' size."""
    D, G, bits, Hkv, P = case["D"], case["G"], case["bits"], case["Hkv"], case["page"]
    codes = torch.empty(pages, Hkv, P, D * bits // 8, dtype=torch.uint8, device=DEV)
    scales = torch.empty(pages, Hkv, P, D // G, dtype=torch.float16, device=DEV)
    step = max(1, (1 << 25) // (Hkv * P * D))
    for a in range(0, pages, step):
        b = min(pages, a + step)
        y = torch.randn(b - a, Hkv, P, D // G, G, generator=g, device=DEV) * spread
        s = (y.abs().amax(-1) / (7 if bits == 4 else 127)).half()
        c = torch.round(y / s.float().unsqueeze(-1)).clamp(-7, 7) if bits == 4 else torch.round(y / s.float().unsqueeze(-1)).clamp(-127, 127)
        c = c.to(torch.int32).reshape(b - a, Hkv, P, D)
        codes[a:b] = ((c[..., 0::2] & 15) | ((c[..., 1::2] & 15) << 4)).to(torch.uint8) if bits == 4 else (c & 255).to(torch.uint8)
        scales[a:b] = s
    return codes, scales


def _seeded(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed((case["mix"] * 1000003 + seed) % (1 << 62))
    return g


def _params(g, D):
    signs = torch.randint(0, 2, (D,), generator=g, device=DEV) * 2 - 1
    lam = torch.exp(0.25 * torch.randn(D, generator=g, device=DEV))
    return signs.to(torch.int8), lam


def _handle(case, signs, lam):
    import rotated_int4_kv_b200 as kvq
    return kvq.Plan(signs.cpu().numpy(), lam.cpu().numpy(), group=case["G"], transform=case["xf"], bits=case["bits"])


def prepare(case, seed):
    g = _seeded(case, seed)
    st = {"case": case}
    if case["op"] == "plan":
        kv, q = _lens(case)
        P, B = case["page"], case["B"]
        most = max(-(-(a + b) // P) for a, b in zip(kv, q)) + 2
        have = [-(-a // P) for a in kv]
        new = sum(-(-(a + b) // P) - h for a, b, h in zip(kv, q, have))
        total = sum(have) + new + 64
        perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
        table = torch.full((B, most), -1, dtype=torch.int32, device=DEV)
        col = torch.arange(most, device=DEV)
        mask = col[None, :] < torch.tensor(have, device=DEV)[:, None]
        table[mask] = perm[: sum(have)]
        taken = 5
        free = perm[sum(have) - taken:] if sum(have) >= taken else torch.cat([perm[:taken], perm[sum(have):]])
        if case["tight"]:
            free = free[: taken + max(1, int(0.8 * new))]
        st.update(kv_lens=torch.tensor(kv, dtype=torch.int32, device=DEV), q_lens=torch.tensor(q, dtype=torch.int32, device=DEV),
                  table=table, free=free.contiguous(), head=torch.tensor([taken], dtype=torch.int32, device=DEV), n=sum(q) + 13)
        if own:
            # what a serving loop keeps between steps: the outputs' buffers
            import rotated_int4_kv_b200 as kvq
            st["out"] = kvq.PagePlan.empty(B, st["n"], DEV)
            st["head_out"] = torch.empty_like(st["head"])
        return st
    D, Hkv, P = case["D"], case["Hkv"], case["page"]
    st["sk"], st["lk"] = _params(g, D)
    st["sv"], st["lv"] = _params(g, D)
    st["Q"] = _basis(D, case["xf"], DEV)            # a program keeps the rotation, as it keeps signs and lambda
    if own:
        # the transform handles that a program makes once per layer (the plain form takes signs and lambda)
        st["pk"], st["pv"] = _handle(case, st["sk"], st["lk"]), _handle(case, st["sv"], st["lv"])
    if case["op"] in ("store", "fetch"):
        n, pad = case["n"], case["pad"]
        pages = -(-n // P) + 3
        # tokens in order within their pages, the pages in any order, as block tables give them
        order = torch.randperm(pages, generator=g, device=DEV)
        t = torch.arange(n, device=DEV)
        slots = (order[t // P] * P + t % P).to(torch.int32)
        st["slots"] = torch.cat([slots, torch.full((pad,), -1, dtype=torch.int32, device=DEV)])
        if case["op"] == "fetch":
            st["kc"], st["ks"] = _packed(g, pages, case, 1.0)
            return st
        # K and V as views into one fused projection, rows of different size, K with a few strong channels
        x = torch.randn(n + pad, 3 * Hkv, D, generator=g, device=DEV)
        x[:, Hkv:2 * Hkv, :4] *= 4.0
        x = (x * torch.exp(0.3 * torch.randn(n + pad, 3 * Hkv, 1, generator=g, device=DEV))).half()
        st["k"], st["v"] = x[:, Hkv:2 * Hkv], x[:, 2 * Hkv:]
        for name in ("k", "v"):
            st[name + "c"] = torch.zeros(pages, Hkv, P, D * case["bits"] // 8, dtype=torch.uint8, device=DEV)
            st[name + "s"] = torch.zeros(pages, Hkv, P, D // case["G"], dtype=torch.float16, device=DEV)
        return st
    kv, q = _lens(case)
    B, Hq = case["B"], case["Hq"]
    need = [-(-a // P) for a in kv]
    pages = sum(need) + 3
    st["kc"], st["ks"] = _packed(g, pages, case, 1.0)
    st["vc"], st["vs"] = _packed(g, pages, case, 1.0)
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(B, max(need) + 1, dtype=torch.int32, device=DEV)
    table[torch.arange(max(need) + 1, device=DEV)[None, :] < torch.tensor(need, device=DEV)[:, None]] = order[: sum(need)]
    st["table"] = table
    st["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
    starts = [0]
    for n in q:
        starts.append(starts[-1] + n)
    st["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    st["q_hi"], st["L"] = max(q), max(kv)
    # queries as a view into one fused projection; of a size that gives some rows a few strong scores
    qkv = (1.5 * torch.randn(starts[-1], Hq + 2 * Hkv, D, generator=g, device=DEV)).half()
    st["q"] = qkv[:, :Hq]
    if own:
        import rotated_int4_kv_b200 as kvq
        # the workspace of a serving loop, allocated once
        st["ws"] = kvq.make_paged_workspace(B, Hq, Hkv, D, starts[-1], st["q_hi"], device=DEV)
    return st


# --------------------------------------------------------------------------- the plain forms
def _plan_plain(st, P):
    kv, q, table, free = st["kv_lens"].long(), st["q_lens"].long(), st["table"], st["free"]
    head, n, M = st["head"].long(), st["n"], table.shape[1]
    have, want = (kv + P - 1) // P, (kv + q + P - 1) // P
    fits = want <= M
    need = torch.where(fits, want - have, 0)
    upto = torch.cumsum(need, 0)
    room = free.shape[0] - head
    served = fits & ((need == 0) | (upto <= room))
    first = upto - need
    starts = torch.cat([torch.zeros(1, dtype=torch.int64, device=q.device), torch.cumsum(q, 0)])
    t = torch.arange(n, device=q.device)
    b = torch.searchsorted(starts[1:], t, right=True).clamp(max=q.shape[0] - 1)
    pos = kv[b] + t - starts[b]
    real = t < starts[-1]
    blk = pos // P
    old = table[b, blk.clamp(max=M - 1)].long()
    taken = free[(head + first[b] + blk - have[b]).clamp(0, free.shape[0] - 1)].long()
    page = torch.where(blk < have[b], old, taken)
    good = real & served[b]
    slots = torch.where(good, page * P + pos % P, -1).int()
    positions = torch.where(real, pos, -1).int()
    col = torch.arange(M, device=q.device)
    fresh = served[:, None] & (col >= have[:, None]) & (col < want[:, None])
    new = free[(head + first[:, None] + col - have[:, None]).clamp(0, free.shape[0] - 1)]
    got = torch.where(served, need, 0).sum()
    info = torch.stack([starts[-1], got, (~served).sum(), need.sum()])
    return {"slots": slots, "positions": positions, "q_starts": starts.int(), "kv_lens": torch.where(served, kv + q, kv).int(),
            "table": torch.where(fresh, new, table), "head": (head + got).int(), "info": info.int()}


def _values(codes, scales, case, dtype=torch.float32):
    """Rows of codes and scales as the rotated values they stand for."""
    c = codes.to(torch.int32)
    if case["bits"] == 4:
        c = torch.stack([c & 15, c >> 4], -1).reshape(*codes.shape[:-1], case["D"])
        c = c - 16 * (c >> 3)
    else:
        c = c - 256 * (c >> 7)
    c = c.to(dtype).reshape(*codes.shape[:-1], case["D"] // case["G"], case["G"])
    return (c * scales.to(dtype).unsqueeze(-1)).reshape(*codes.shape[:-1], case["D"])


def _rows(pages, slots, P):
    """Rows [n, kv heads, ...] of the pages at `slots`."""
    s = slots.long().clamp(min=0)
    return pages[s // P, :, s % P]


def _decode_plain(codes, scales, slots, signs, lam, Q, case):
    y = _values(_rows(codes, slots, case["page"]), _rows(scales, slots, case["page"]), case)
    x = (y / lam) @ Q.float() * signs.float()
    return torch.where((slots >= 0)[:, None, None], x, 0.0).half()


def _encode_plain(x, codes, scales, slots, signs, lam, Q, case):
    """In 64 bits up to the rounding: a value next to a border falls on the side it belongs to."""
    D, G, P, top = case["D"], case["G"], case["page"], 7 if case["bits"] == 4 else 127
    live = slots >= 0
    y = (((x[live].double() * signs.double()) @ Q.T) * lam.double()).reshape(-1, x.shape[1], D // G, G)
    s = (y.abs().amax(-1) / top).clamp(max=65504.0).half()
    c = torch.where(s.unsqueeze(-1) > 0, torch.round(y / s.double().unsqueeze(-1)), 0.0).clamp(-top, top)
    c = c.to(torch.int32).reshape(-1, x.shape[1], D)
    c = ((c[..., 0::2] & 15) | ((c[..., 1::2] & 15) << 4)) if case["bits"] == 4 else c & 255
    at = slots[live].long()
    codes[at // P, :, at % P] = c.to(torch.uint8)
    scales[at // P, :, at % P] = s


def _attend_plain(st, case):
    """Padded to the longest request: pages gathered, decoded to the rows' own domain, masked softmax attention."""
    D, Hq, Hkv, P, B, W = case["D"], case["Hq"], case["Hkv"], case["page"], case["B"], case["window"]
    table = st["table"].long()
    M = -(-st["L"] // P)

    def rows(codes, scales, signs, lam):
        at = table[:, :M]
        y = _values(codes[at].transpose(1, 2).reshape(B, Hkv, M * P, -1), scales[at].transpose(1, 2).reshape(B, Hkv, M * P, -1), case)
        return (y / lam) @ st["Q"].float() * signs.float()

    K, V = rows(st["kc"], st["ks"], st["sk"], st["lk"]), rows(st["vc"], st["vs"], st["sv"], st["lv"])
    starts, kv = st["starts"].long(), st["kv_lens"].long()
    n = starts[1:] - starts[:-1]
    j = torch.arange(st["q_hi"], device=K.device)
    inside = j[None, :] < n[:, None]
    at = (starts[:-1, None] + j[None, :]).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][at].float().reshape(B, -1, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)            # [B, Hkv, G, Q, D]
    s = torch.matmul(q.reshape(B, Hkv, -1, D), K.transpose(-1, -2)).reshape(*q.shape[:4], -1) / math.sqrt(D)
    t = torch.arange(K.shape[2], device=K.device)
    pos = (kv - n)[:, None] + j[None, :]
    ok = t[None, None, :] <= pos[:, :, None]
    if W:
        ok = ok & (t[None, None, :] > pos[:, :, None] - W)
    s = s.masked_fill_(~ok[:, None, None], -math.inf)
    p = torch.exp_(s.sub_(s.amax(-1, keepdim=True)))
    o = torch.matmul(p.reshape(B, Hkv, -1, p.shape[-1]), V).reshape(*q.shape) / p.sum(-1, keepdim=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, -1, Hq, D)
    return o[inside].half()


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import rotated_int4_kv_b200 as kvq
        if op == "plan":
            p = kvq.page_plan(state["kv_lens"], state["q_lens"], state["table"], state["free"], state["head"], case["page"],
                              out=state["out"], free_head_out=state["head_out"])
            return {"slots": p.slots, "positions": p.positions, "q_starts": p.q_starts, "kv_lens": p.kv_lens,
                    "table": state["table"], "head": state["head_out"], "info": p.info}
        if op == "store":
            kvq.encode_paged([(state["pk"], state["k"], state["kc"], state["ks"]), (state["pv"], state["v"], state["vc"], state["vs"])],
                             state["slots"])
            return {"k": kvq.decode_paged(state["pk"], state["kc"], state["ks"], state["slots"]),
                    "v": kvq.decode_paged(state["pv"], state["vc"], state["vs"], state["slots"])}
        if op == "fetch":
            return kvq.decode_paged(state["pk"], state["kc"], state["ks"], state["slots"])
        return kvq.attend_paged(state["pk"], state["pv"], state["q"], state["kc"], state["ks"], state["vc"], state["vs"],
                                state["table"], state["kv_lens"], q_starts=state["starts"], max_q_len=state["q_hi"],
                                max_kv_len=state["L"], window=case["window"], workspace=state["ws"])
    if op == "plan":
        return _plan_plain(state, case["page"])
    if op == "store":
        _encode_plain(state["k"], state["kc"], state["ks"], state["slots"], state["sk"], state["lk"], state["Q"], case)
        _encode_plain(state["v"], state["vc"], state["vs"], state["slots"], state["sv"], state["lv"], state["Q"], case)
        return {"k": _decode_plain(state["kc"], state["ks"], state["slots"], state["sk"], state["lk"], state["Q"], case),
                "v": _decode_plain(state["vc"], state["vs"], state["slots"], state["sv"], state["lv"], state["Q"], case)}
    if op == "fetch":
        return _decode_plain(state["kc"], state["ks"], state["slots"], state["sk"], state["lk"], state["Q"], case)
    return _attend_plain(state, case)


# --------------------------------------------------------------------------- 64 bits, from the definition
def exact(case, seed):
    if case["op"] == "plan":
        return None
    st = prepare(case, seed)
    D, P = case["D"], case["page"]
    Q = _basis(D, case["xf"], DEV)

    def back(codes, scales, slots, signs, lam):
        """x = s * Q^T (c * scale / lambda), row by row."""
        at = slots.long()
        y = _values(codes[at // P, :, at % P], scales[at // P, :, at % P], case, torch.float64)
        return torch.einsum("nhc,cd->nhd", y / lam.double(), Q) * signs.double()

    if case["op"] == "fetch":
        out = torch.zeros(st["slots"].shape[0], case["Hkv"], D, dtype=torch.float64, device=DEV)
        out[: case["n"]] = back(st["kc"], st["ks"], st["slots"][: case["n"]], st["sk"], st["lk"])
        return out
    if case["op"] == "store":
        res = {}
        top = 7.0 if case["bits"] == 4 else 127.0
        for name, signs, lam in (("k", st["sk"], st["lk"]), ("v", st["sv"], st["lv"])):
            x = st[name][: case["n"]].double()
            y = torch.einsum("nhd,cd->nhc", x * signs.double(), Q) * lam.double()
            yg = y.unflatten(-1, (D // case["G"], case["G"]))
            sc = torch.minimum(yg.abs().max(-1).values / top, torch.tensor(65504.0, dtype=torch.float64, device=DEV)).half().double()
            c = torch.where(sc[..., None] == 0, torch.zeros_like(yg), torch.round(yg / sc[..., None])).clip(-top, top)
            xh = torch.einsum("nhc,cd->nhd", (c * sc[..., None]).flatten(-2) / lam.double(), Q) * signs.double()
            res[name] = torch.cat([xh, torch.zeros(case["pad"], *xh.shape[1:], dtype=torch.float64, device=DEV)])
        return res
    kv, q = _lens(case)
    Hq, Hkv, W = case["Hq"], case["Hkv"], case["window"]
    if sum(a * b for a, b in zip(kv, q)) * Hq * D > 1 << 42:
        return None
    out = torch.empty(sum(q), Hq, D, dtype=torch.float64, device=DEV)
    at0 = 0
    for b, (L, n) in enumerate(zip(kv, q)):
        t = torch.arange(L, device=DEV)
        slots = st["table"][b].long()[t // P] * P + t % P
        K, V = back(st["kc"], st["ks"], slots, st["sk"], st["lk"]), back(st["vc"], st["vs"], slots, st["sv"], st["lv"])
        pos = torch.arange(L - n, L, device=DEV)
        hide = t[None, :] > pos[:, None]
        if W:
            hide = hide | (t[None, :] <= pos[:, None] - W)
        for h in range(Hq):
            z = st["q"][at0:at0 + n, h].double() @ K[:, h // (Hq // Hkv)].T / math.sqrt(D)
            z = torch.where(hide, -math.inf, z)
            out[at0:at0 + n, h] = torch.softmax(z, -1) @ V[:, h // (Hq // Hkv)]
        at0 += n
    return out
