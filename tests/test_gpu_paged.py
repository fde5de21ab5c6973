"""The paged operators on the GPU against plain 64-bit forms: step planning and page release
(exact), encode into pages, decode from pages, ragged causal attention over pages, and a
serving loop of all of them through PagedInt4KVCache."""
import numpy as np
import pytest

import kvgen
import oracle
from tests import paged_ref
from tests.parity import BOUNDARY_TALLY, check_encode, check_rel_l2

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    import rotated_int4_kv_b200 as k
    return k


@pytest.fixture(autouse=True)
def no_device_errors(kvq):
    yield
    torch.cuda.synchronize()
    assert kvq.poll_device_errors() == 0


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).cuda()


def make_plan(kvq, D, kind, G=32, xf="srft", bits=4, seed=17):
    params = kvgen.plan_params(D, seed=seed, kind=kind)
    return kvq.Plan(*params, G, xf, bits), params


# ---------------------------------------------------------------- step planning
def plan_case(rng, B, P, M, n_free, head, idle=0.2, fresh=0.3, q_hi=40):
    kv = np.where(rng.random(B) < fresh, 0, rng.integers(1, max(2, M * P - 1), B))
    q = np.where(rng.random(B) < idle, 0, np.where(kv == 0, rng.integers(1, q_hi + 1, B), rng.integers(1, 4, B)))
    table = np.full((B, M), -1, np.int32)
    for b in range(B):
        have = -(-int(kv[b]) // P)
        table[b, :have] = rng.integers(0, 5000, have)
    return kv.astype(np.int32), q.astype(np.int32), table, rng.permutation(n_free + 7)[:n_free].astype(np.int32), head


def check_plan(kvq, kv, q, table, free, head, P, n, in_place):
    ref = paged_ref.plan_step(kv, q, table, free, head, P, n)
    wide = torch.full((table.shape[0], table.shape[1] + 3), -9, dtype=torch.int32, device="cuda")
    tab = wide[:, 1:1 + table.shape[1]]  # strided rows, not at the buffer's start
    tab.copy_(torch.from_numpy(table))
    lens, h = i32(kv), i32([head])
    out, h_out = None, None
    if in_place:
        out = kvq.PagePlan.empty(len(kv), n, lens.device)._replace(kv_lens=lens)
    else:
        h_out = torch.empty_like(h)
    got = kvq.page_plan(lens, i32(q), tab, i32(free), h, P, n, out=out, free_head_out=h_out)
    torch.cuda.synchronize()
    for name in ("slots", "positions", "q_starts", "kv_lens", "info"):
        assert np.array_equal(getattr(got, name).cpu().numpy(), ref[name]), name
    assert np.array_equal(tab.cpu().numpy(), ref["table"])
    assert int((h if in_place else h_out).item()) == ref["head"]
    assert (wide[:, 0] == -9).all() and (wide[:, 1 + table.shape[1]:] == -9).all()
    if not in_place:
        assert np.array_equal(lens.cpu().numpy(), kv) and int(h.item()) == head


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,P,M", [(1, 16, 4), (5, 16, 1), (33, 32, 9), (1025, 64, 7), (3000, 128, 3), (16384, 16, 2)])
def test_page_plan(kvq, B, P, M, in_place):
    rng = np.random.default_rng(B)
    for n_free, head, pad in ((4 * B + 50, 3, 13), (B // 3, 0, 0), (7, 7, 5), (9, 20, -2)):
        kv, q, table, free, head = plan_case(rng, B, P, M, n_free, head)
        check_plan(kvq, kv, q, table, free, head, P, max(0, int(q.sum()) + pad), in_place)


def test_page_plan_edges(kvq):
    one = np.array([[5, 6]], np.int32)
    for kv, q in (([0], [0]), ([32], [0]), ([31], [1]), ([32], [1]), ([0], [32]), ([0], [33]), ([-4], [3]), ([7], [-2]),
                  ([2 ** 31 - 1], [2 ** 31 - 1])):
        n = 40 if max(q) < 2 ** 20 else 0
        if n:
            check_plan(kvq, np.array(kv, np.int32), np.array(q, np.int32), one, np.array([8, 9, 10], np.int32), 0, 16, n, False)
        else:  # lengths that fit no table: refused, sums saturate
            got = kvq.page_plan(i32(kv), i32(q), i32(one), i32([8, 9]), i32([0]), 16, 5)
            assert got.slots.tolist() == [-1] * 5 and got.info.tolist() == [2 ** 31 - 1, 0, 1, 0]
            assert got.kv_lens.tolist() == kv and got.q_starts.tolist() == [0, 2 ** 31 - 1]
    # no requests, no free pages
    got = kvq.page_plan(i32([]), i32([]), i32(np.zeros((0, 3))), i32([]), i32([0]), 16, 3)
    assert got.slots.tolist() == [-1] * 3 and got.q_starts.tolist() == [0] and got.info.tolist() == [0, 0, 0, 0]
    # a page number whose slots would pass 32 bits names no slot
    got = kvq.page_plan(i32([3]), i32([1]), i32([[2 ** 28]]), i32([]), i32([0]), 16, 1)
    assert got.slots.tolist() == [-1]


def test_page_release_round_trip(kvq):
    rng = np.random.default_rng(3)
    B, P, M, F = 1500, 16, 4, 9000
    free = rng.permutation(F).astype(np.int32)
    lens, head, fr = i32(np.zeros(B)), i32([0]), i32(free)
    table = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
    held = [[] for _ in range(B)]
    for _ in range(3):
        q = rng.integers(0, 20, B)
        out = kvq.PagePlan.empty(B, int(q.sum()), lens.device)._replace(kv_lens=lens)
        kvq.page_plan(lens, i32(q), table, fr, head, P, out=out)
        t, n = table.cpu().numpy(), lens.cpu().numpy()
        held = [t[b, :-(-int(n[b]) // P)].tolist() for b in range(B)]
        done = rng.random(B) < 0.4
        before = fr.cpu().numpy()[: int(head.item())]
        kvq.page_release(torch.from_numpy(done).cuda(), lens, table, fr, head, P)
        back = [x for b in range(B) if done[b] for x in held[b]]
        h = int(head.item())
        assert h == len(before) - len(back) and (lens.cpu().numpy()[done] == 0).all()
        f = fr.cpu().numpy()
        assert f[h:h + len(back)].tolist() == back[::-1]
        # what is free and what is held are all pages, once each
        live = [x for b in range(B) if not done[b] for x in held[b]]
        assert sorted(f[h:].tolist() + live) == list(range(F))
    # more pages than were taken: those past the list's start are dropped
    head.zero_()
    lens.fill_(P)
    kvq.page_release(torch.ones(B, dtype=torch.bool, device="cuda"), lens, table, fr, head, P)
    assert int(head.item()) == 0 and int(lens.sum().item()) == 0


# ---------------------------------------------------------------- encode, decode
FORMS = [(128, 32, 4, "srft"), (128, 16, 4, "srht"), (256, 32, 4, "srft"), (256, 16, 8, "srht"), (128, 32, 8, "srft"),
         (256, 32, 8, "srft"), (128, 16, 8, "srft"), (256, 16, 4, "srft"), (256, 32, 4, "srht")]


@pytest.mark.parametrize("D,G,bits,xf", FORMS)
@pytest.mark.parametrize("n,H,P,jobs", [(1, 1, 16, 1), (7, 3, 32, 2), (131, 2, 64, 3), (37, 8, 128, 2), (3, 128, 16, 2)])
def test_encode_decode_paged(kvq, D, G, bits, xf, n, H, P, jobs):
    rng = np.random.default_rng(n * H + D)
    pages = -(-n // P) + 2
    slots = rng.permutation(pages * P)[:n].astype(np.int32)
    if n > 2:
        slots[1], slots[n - 1] = -1, pages * P      # a padded token and one past the pages
    use = (slots >= 0) & (slots < pages * P)
    wl = kvgen.WORKLOADS["qwen" if D == 128 else "gemma"]
    made, arg = [], []
    for j in range(jobs):
        plan, params = make_plan(kvq, D, "k", G, xf, bits, seed=5 + j)
        x = kvgen.kv_numpy(wl, "k", (1, H, n, D), seed=9 + j)[0].transpose(1, 0, 2)    # [n, H, D]
        wide = torch.full((n, H + 1, D + 8), float("nan"), dtype=torch.float16, device="cuda")
        view = wide[:, 1:, :D]
        view.copy_(torch.from_numpy(np.ascontiguousarray(x)))
        codes = torch.full((pages, H, P, D * bits // 8), 0xA5, dtype=torch.uint8, device="cuda")
        scales = torch.full((pages, H, P, D // G), 7.0, dtype=torch.float16, device="cuda")
        made.append((x, params, codes, scales))
        arg.append((plan, view, codes, scales))
    kvq.encode_paged(arg, i32(slots))
    torch.cuda.synchronize()
    for (x, params, codes, scales), (plan, *_) in zip(made, arg):
        c, s = codes.cpu().numpy(), scales.cpu().numpy()
        bad, total = check_encode(x[use], *params, G, paged_ref.rows_at(c, slots[use], P),
                                  paged_ref.rows_at(s, slots[use], P), count_only=True, transform=xf, bits=bits)
        if bits == 4:
            BOUNDARY_TALLY["bad"] += bad
            BOUNDARY_TALLY["all"] += total
        rest = np.ones((pages, P), bool)
        rest[slots[use] // P, slots[use] % P] = False
        assert (c.transpose(0, 2, 1, 3)[rest] == 0xA5).all() and (s.transpose(0, 2, 1, 3)[rest] == 7.0).all()
        # read back: any order, repeats, slots that name nothing
        look = np.concatenate([slots[::-1], slots[:1], np.array([-1, pages * P, 2 ** 31 - 1], np.int32)])
        out = kvq.decode_paged(plan, codes, scales, i32(look)).cpu().numpy().astype(np.float64)
        live = (look >= 0) & (look < pages * P)
        ref = paged_ref.decoded(c, s, look[live], P, params, G, xf, bits)
        check_rel_l2(out[live].reshape(-1, D), ref.reshape(-1, D), label="decode_paged")
        assert (out[~live] == 0).all()


def test_encode_paged_matches_the_dense_encode(kvq):
    D, H, n, P = 128, 4, 96, 32
    plan, _ = make_plan(kvq, D, "v")
    x = torch.randn(n, H, D, device="cuda").half()
    dc = torch.zeros(1, H, n, D // 2, dtype=torch.uint8, device="cuda")
    ds = torch.zeros(1, H, n, D // 32, dtype=torch.float16, device="cuda")
    kvq.set_encode_path("tensor")
    try:
        kvq.encode(plan, x.transpose(0, 1)[None].contiguous(), dc, ds, 0)
    finally:
        kvq.set_encode_path("auto")
    pc = torch.zeros(3, H, P, D // 2, dtype=torch.uint8, device="cuda")
    ps = torch.zeros(3, H, P, D // 32, dtype=torch.float16, device="cuda")
    kvq.encode_paged([(plan, x, pc, ps)], torch.arange(n, dtype=torch.int32, device="cuda"))
    assert torch.equal(pc.transpose(0, 1).reshape(H, n, -1), dc[0]) and torch.equal(ps.transpose(0, 1).reshape(H, n, -1), ds[0])


# ---------------------------------------------------------------- attention
def random_pages(rng, pages, H, P, D, G, bits):
    codes = rng.integers(-oracle.qmax(bits), oracle.qmax(bits) + 1, (pages, H, P, D)).astype(np.int8)
    scales = (rng.uniform(0.5, 1.5, (pages, H, P, D // G)) / oracle.qmax(bits)).astype(np.float16)
    return oracle.pack_codes(codes, bits).view(np.uint8).reshape(pages, H, P, D * bits // 8), scales


class Cache:
    """Pages, tables and queries of one attention call; what no request attends is set to NaN scales."""

    def __init__(self, kvq, kv, q, Hq, Hkv, D, G, bits, xf, P, seed=0, pad=0, q_size=1.0, spoil=True):
        rng = np.random.default_rng(seed)
        self.kv, self.q_lens, self.form = list(kv), list(q), (G, xf, bits)
        self.P, B = P, len(kv)
        need = [-(-L // P) for L in kv]
        pages = sum(need) + 2
        order = rng.permutation(pages).astype(np.int32)
        self.M = max(need + [1]) + 1
        self.table = np.full((B, self.M), -7, np.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = order[at:at + m]
            at += m
        self.kc, self.ks = random_pages(rng, pages, Hkv, P, D, G, bits)
        self.vc, self.vs = random_pages(rng, pages, Hkv, P, D, G, bits)
        if spoil:
            held = np.zeros((pages, P), bool)
            for b, L in enumerate(kv):
                t = np.arange(L)
                held[self.table[b][t // P], t % P] = True
            for s in (self.ks, self.vs):
                s.transpose(0, 2, 1, 3)[~held] = np.nan
        n = sum(q)
        self.q = (q_size * rng.standard_normal((n, Hq, D))).astype(np.float16)
        self.pk, self.kp = make_plan(kvq, D, "k", G, xf, bits)
        self.pv, self.vp = make_plan(kvq, D, "v", G, xf, bits)
        self.starts = i32(np.concatenate([[0], np.cumsum(q)]))
        wide = torch.zeros((n + pad, Hq + 2, D + 8), dtype=torch.float16, device="cuda")
        wide[:n, 1:1 + Hq, :D] = torch.from_numpy(self.q).cuda()
        self.qd = wide[:, 1:1 + Hq, :D]
        self.dev = [torch.from_numpy(a).cuda() for a in (self.kc, self.ks, self.vc, self.vs)]
        self.tab, self.lens = i32(self.table), i32(kv)

    def run(self, kvq, starts=True, **kw):
        return kvq.attend_paged(self.pk, self.pv, self.qd, *self.dev, self.tab, self.lens, self.starts if starts else None,
                                **kw)

    def ref(self, window=0, sigma=None):
        return paged_ref.attend(self.q, self.kc, self.ks, self.vc, self.vs, self.table, self.kv, self.q_lens, self.kp,
                                self.vp, *self.form, window=window, sigma=sigma)

    def check(self, got, window=0, sigma=None, tol=2e-3, label=""):
        D = self.q.shape[2]
        ref = self.ref(window, sigma)
        got = got.detach().cpu().numpy()[: len(ref)].astype(np.float64)
        empty = (ref == 0).all(-1)
        assert (got[empty] == 0).all(), label
        check_rel_l2(got[~empty].reshape(-1, D), ref[~empty].reshape(-1, D), tol=tol, label=label)


HEADS = [(12, 2, 128), (32, 8, 128), (8, 1, 128), (4, 1, 256), (3, 3, 128), (2, 2, 256)]


@pytest.mark.parametrize("G,bits,xf", [(32, 4, "srft"), (16, 4, "srht"), (32, 8, "srht"), (16, 8, "srft")])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_attend_paged_single_tokens(kvq, Hq, Hkv, D, G, bits, xf):
    for seed, (P, kv) in enumerate(((16, [1, 17, 300]), (64, [63, 64, 65, 1000, 2]), (128, [129]), (32, [0, 31, 0]))):
        c = Cache(kvq, kv, [1] * len(kv), Hq, Hkv, D, G, bits, xf, P, seed=seed)
        c.check(c.run(kvq, starts=False), label=f"P {P} kv {kv}")
        c.check(c.run(kvq, window=40), window=40, label=f"window, P {P}")


@pytest.mark.parametrize("G,bits,xf", [(32, 4, "srft"), (16, 4, "srft"), (32, 8, "srft"), (16, 8, "srht")])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_attend_paged_several_tokens(kvq, Hq, Hkv, D, G, bits, xf):
    for seed, (P, kv, q, w) in enumerate(((16, [5, 200, 77], [5, 3, 1], 0), (32, [300, 9, 40], [7, 0, 6], 33),
                                          (128, [257], [9], 130), (16, [3, 50], [6, 2], 0))):
        c = Cache(kvq, kv, q, Hq, Hkv, D, G, bits, xf, P, seed=seed, pad=2)
        out = torch.full((sum(q) + 2, Hq, D), 5.0, dtype=torch.float16, device="cuda")
        c.check(c.run(kvq, max_q_len=max(q), window=w, out=out), window=w, label=f"kv {kv} q {q} window {w}")
        assert (out[sum(q):] == 5.0).all()   # rows of no request stay


@pytest.mark.parametrize("G,bits,xf", [(32, 4, "srft"), (16, 4, "srht"), (32, 8, "srht"), (16, 8, "srft")])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_attend_paged_prompts(kvq, Hq, Hkv, D, G, bits, xf):
    """Prompts and chunks of prompts: many query tokens, lengths off the tiles' borders."""
    for seed, (P, kv, q, w) in enumerate(((64, [130, 70], [130, 33], 0), (16, [400], [65], 100), (32, [40, 150, 1], [40, 90, 1], 17),
                                          (128, [333, 600], [300, 0], 0))):
        c = Cache(kvq, kv, q, Hq, Hkv, D, G, bits, xf, P, seed=seed, pad=3)
        out = torch.full((sum(q) + 3, Hq, D), 5.0, dtype=torch.float16, device="cuda")
        c.check(c.run(kvq, max_q_len=max(q), window=w, out=out), window=w, label=f"kv {kv} q {q} window {w}")
        assert (out[sum(q):] == 5.0).all()


@pytest.mark.parametrize("B", [300, 1300])
def test_attend_paged_many_requests(kvq, B):
    rng = np.random.default_rng(B)
    kv = rng.integers(0, 40, B)
    c = Cache(kvq, kv, [1] * B, 4, 1, 128, 32, 4, "srft", 16, seed=2)
    c.check(c.run(kvq, starts=False))
    q = rng.integers(0, 3, B)
    c = Cache(kvq, kv, q, 4, 1, 128, 32, 4, "srft", 16, seed=3)
    c.check(c.run(kvq, max_q_len=2))
    q = np.where(rng.random(B) < 0.05, 30, q)
    c = Cache(kvq, kv, q, 4, 1, 128, 32, 4, "srft", 16, seed=4)
    c.check(c.run(kvq, max_q_len=30))


def test_attend_paged_long_ragged_batch(kvq):
    for Hq, Hkv, D, kv, P in ((32, 8, 128, [9000, 3, 500], 64), (4, 1, 256, [20001, 4097], 16)):
        c = Cache(kvq, kv, [1] * len(kv), Hq, Hkv, D, 32, 4, "srft", P)
        c.check(c.run(kvq, starts=False))
        c.check(c.run(kvq, starts=False, window=300, softmax_scale=0.03), window=300, sigma=0.03)
    c = Cache(kvq, [7000, 50], [100, 50], 8, 2, 128, 32, 4, "srft", 32)
    c.check(c.run(kvq, max_q_len=100))


def test_attend_paged_length_bounds(kvq):
    """kv_lens past max_kv_len or the table are cut; query tokens past max_q_len get no output."""
    c = Cache(kvq, [100, 40], [1, 1], 4, 1, 128, 32, 4, "srft", 16)
    c.lens = i32([250, 40])       # 250 exceeds the table's (7 + 1) pages of 16: cut to max_kv_len = 100
    c.check(c.run(kvq, starts=False, max_kv_len=100))
    c = Cache(kvq, [100, 40], [6, 2], 4, 1, 128, 32, 4, "srft", 16)
    out = torch.full((8, 4, 128), 5.0, dtype=torch.float16, device="cuda")
    c.run(kvq, max_q_len=4, out=out)
    full = torch.full_like(out, 5.0)
    c.run(kvq, max_q_len=6, out=full)
    assert (out[4:6] == 5.0).all()
    assert torch.equal(out[:4], full[:4]) and torch.equal(out[6:], full[6:])
    # more query tokens than the request holds: those before its first token attend nothing
    c = Cache(kvq, [3], [5], 4, 1, 128, 32, 4, "srft", 16)
    c.check(c.run(kvq, max_q_len=5))


def test_attend_paged_bad_pages_raise_a_flag(kvq):
    c = Cache(kvq, [100], [1], 4, 1, 128, 32, 4, "srft", 16, spoil=False)
    for bad in (-1, 10 ** 6):
        c.tab[0, 3] = bad
        got = c.run(kvq, starts=False)
        torch.cuda.synchronize()
        assert kvq.poll_device_errors() == 8 and torch.isfinite(got).all()
    # entries without an attended token are not looked at (-7 behind the last page; in front of the window)
    c = Cache(kvq, [100], [1], 4, 1, 128, 32, 4, "srft", 16)
    c.tab[0, :4] = -1
    c.check(c.run(kvq, starts=False, window=20), window=20)
    c = Cache(kvq, [500], [100], 4, 1, 128, 32, 4, "srft", 16)
    c.tab[0, :20] = -1
    c.check(c.run(kvq, max_q_len=100, window=40), window=40)


def test_attend_paged_extreme_scales(kvq):
    """V and K scales over fp16's whole range: the products stay within the kernels' number formats."""
    for q, kv in (([1], [300]), ([90], [300])):
        for vs, ksz in ((9000.0, 1.0), (6e-7, 1.0), (1.0, 3e4)):
            c = Cache(kvq, kv, q, 4, 1, 128, 32, 4, "srft", 16, seed=5, q_size=1.0 / ksz)
            c.vs = (c.vs.astype(np.float32) * vs).astype(np.float16)
            c.ks = np.minimum(c.ks.astype(np.float32) * ksz, 65504).astype(np.float16)
            c.dev[1], c.dev[3] = torch.from_numpy(c.ks).cuda(), torch.from_numpy(c.vs).cuda()
            ref = c.ref()
            got = c.run(kvq, max_q_len=q[0]).cpu().numpy()
            fits = np.abs(ref) < 6e4
            big = np.where(fits, ref, 0)
            # fp16 outputs: half a step is at least 2^-25, whatever the value
            err = np.abs(np.where(fits, got, 0) - big)
            assert (err <= 4e-3 * np.abs(big).max(-1, keepdims=True) + 2.0 ** -24).all()


def test_attend_paged_workspace_serves_any_geometry(kvq):
    """One workspace for calls of different head sizes and counts, one after another."""
    cs = [Cache(kvq, [900, 33], [1, 1], *h, 32, 4, "srft", 16) for h in HEADS]
    cs += [Cache(kvq, [900, 333], [60, 150], *h, 32, 4, "srft", 16) for h in HEADS[:4]]
    n = max(kvq.paged_workspace_size(2, h[0], h[1], h[2], 400, 400) for h in HEADS)
    ws = torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")   # any contents will do
    for _ in range(2):
        for c in cs:
            c.check(c.run(kvq, max_q_len=max(c.q_lens), workspace=ws))
    with pytest.raises(kvq.KvqError):
        cs[0].run(kvq, max_q_len=1, workspace=ws[:64])


def test_attend_paged_is_deterministic_and_captures(kvq):
    for q in ([1, 1, 1], [40, 1, 25]):
        c = Cache(kvq, [3000, 41, 777], q, 12, 2, 128, 32, 4, "srft", 16)
        want = c.run(kvq, max_q_len=max(q))
        ws = kvq.make_paged_workspace(3, 12, 2, 128, sum(q), max(q))
        out = torch.empty_like(want)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            c.run(kvq, max_q_len=max(q), workspace=ws, out=out)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(kvq, max_q_len=max(q), workspace=ws, out=out)
            c.run(kvq, max_q_len=max(q), workspace=ws, out=out)
        for _ in range(3):
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
        # new lengths in place: the captured call follows them
        c.kv[0] = 1500
        c.lens[0] = 1500
        g.replay()
        c.check(out)


def test_attend_paged_stream_argument(kvq):
    c = Cache(kvq, [600, 70], [1, 1], 8, 1, 128, 32, 4, "srft", 16)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = c.run(kvq, starts=False, stream=s)
    s.synchronize()
    c.check(got)


def test_paged_refusals(kvq):
    c = Cache(kvq, [40, 20], [1, 1], 4, 1, 128, 32, 4, "srft", 16)
    other, _ = make_plan(kvq, 128, "v", bits=8)
    p256, _ = make_plan(kvq, 256, "v")
    kc, ks, vc, vs = c.dev
    for call in (lambda: kvq.attend_paged(c.pk, c.pv, c.qd[:1], *c.dev, c.tab, c.lens),                 # n != B
                 lambda: kvq.attend_paged(c.pk, c.pv, c.qd.float(), *c.dev, c.tab, c.lens),
                 lambda: kvq.attend_paged(c.pk, c.pv, c.qd, kc, ks, vc[:1], vs[:1], c.tab, c.lens),
                 lambda: kvq.attend_paged(c.pk, c.pv, c.qd, kc, vs[..., :2], vc, vs, c.tab, c.lens),
                 lambda: kvq.attend_paged(c.pk, c.pv, c.qd, *c.dev, c.tab[:1], c.lens),
                 lambda: kvq.attend_paged(c.pk, c.pv, c.qd, *c.dev, c.tab.long(), c.lens),
                 lambda: kvq.attend_paged(c.pk, p256, c.qd, *c.dev, c.tab, c.lens),
                 lambda: kvq.attend_paged(c.pk, other, c.qd, *c.dev, c.tab, c.lens),
                 lambda: kvq.attend_paged(c.pk, c.pv, c.qd, *c.dev, c.tab, c.lens, c.starts[:2]),
                 lambda: c.run(kvq, window=-1), lambda: c.run(kvq, max_q_len=0), lambda: c.run(kvq, max_kv_len=-1),
                 lambda: kvq.attend_paged(c.pk, c.pv, torch.zeros(2, 4, 132, dtype=torch.float16, device="cuda")[..., 4:],
                                          *c.dev, c.tab, c.lens),                                       # alignment
                 lambda: kvq.decode_paged(c.pk, kc, ks, c.lens.long()),
                 lambda: kvq.decode_paged(other, kc, ks, c.lens),
                 lambda: kvq.encode_paged([(c.pk, torch.zeros(2, 2, 128, dtype=torch.float16, device="cuda"), kc, ks)], c.lens),
                 lambda: kvq.encode_paged([(c.pk, torch.zeros(1, 1, 128, dtype=torch.float16, device="cuda").expand(2, 1, 128),
                                            kc, ks)], c.lens)):                                         # overlapping rows
        with pytest.raises((ValueError, TypeError, kvq.KvqError)):
            call()


# ---------------------------------------------------------------- all of them together
@pytest.mark.parametrize("Hq,Hkv,D,P,bits", [(8, 2, 128, 16, 4), (4, 1, 256, 32, 4), (4, 4, 128, 64, 8)])
def test_paged_cache_serves_ragged_requests(kvq, Hq, Hkv, D, P, bits):
    """Requests come, grow, end and give their pages back; every step's attention is checked
    against the formula on what the pages then hold, and the pages against the tokens stored."""
    rng = np.random.default_rng(D + P)
    B, L, M = 4, 2, 8
    kp = [kvgen.plan_params(D, seed=3, layer=l, kind="k") for l in range(L)]
    vp = [kvgen.plan_params(D, seed=3, layer=l, kind="v") for l in range(L)]
    cache = kvq.PagedInt4KVCache(L, B, Hkv, D, 14, P, M, kp, vp, bits=bits)
    length, texts = [0] * B, [[] for _ in range(B)]   # per request: stored K of layer 0
    taken = 0
    for step_no in range(9):
        q = [int(rng.choice([0, 1, 1, 3, int(1.7 * P)])) if length[b] == 0 or step_no % 3 else 1 for b in range(B)]
        n = sum(q) + 2
        ref = paged_ref.plan_step(length, q, cache.block_table.cpu().numpy(), cache.free_pages.cpu().numpy(),
                                  int(cache.free_head.item()), P, n)
        step = cache.begin(i32(q), n)
        assert np.array_equal(step.slots.cpu().numpy(), ref["slots"])
        assert np.array_equal(cache.block_table.cpu().numpy(), ref["table"])
        assert np.array_equal(cache.kv_lens.cpu().numpy(), ref["kv_lens"])
        served = [ref["kv_lens"][b] == length[b] + q[b] for b in range(B)]
        length = ref["kv_lens"].tolist()
        at = 0
        x = rng.standard_normal((L, 2, n, Hkv, D)).astype(np.float16)
        for b in range(B):
            if served[b]:
                texts[b] += list(x[0, 0, at:at + q[b]])
            at += q[b]
        for l in range(L):
            cache.update(l, *torch.from_numpy(x[l]).cuda(), step)
            qs = rng.standard_normal((n, Hq, D)).astype(np.float16)
            out = torch.zeros((n, Hq, D), dtype=torch.float16, device="cuda")
            cache.attend(l, torch.from_numpy(qs).cuda(), step, max_q_len=max(q + [1]), out=out)
            got = out.cpu().numpy().astype(np.float64)
            pages = [t[l].cpu().numpy() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
            want = paged_ref.attend(qs, *pages, ref["table"], length, q, kp[l], vp[l], 32, "srft", bits)
            at = 0
            for b in range(B):  # refused requests' tokens have no place: whatever they read is not checked
                if served[b] and q[b]:
                    check_rel_l2(got[at:at + q[b]].reshape(-1, D), want[at:at + q[b]].reshape(-1, D), label=f"step {step_no}")
                at += q[b]
            assert (got[sum(q):] == 0).all()
        for b in range(B):
            if length[b]:
                t = np.arange(length[b])
                slots = i32(ref["table"][b][t // P] * P + t % P)
                back = kvq.decode_paged(cache.k_plans[0], cache.k_codes[0], cache.k_scales[0], slots).cpu().numpy()
                x0 = np.stack(texts[b]).astype(np.float64)
                # quantising by 1/7 (1/127) of the group's largest value: rms error about 0.29 steps of it
                assert np.linalg.norm(back - x0) < (0.2 if bits == 4 else 0.012) * np.linalg.norm(x0)
        done = rng.random(B) < 0.3
        cache.release(torch.from_numpy(done).cuda())
        for b in range(B):
            if done[b]:
                length[b], texts[b] = 0, []
        taken = int(cache.free_head.item())
        assert taken == sum(-(-n // P) for n in length)


# ---------------------------------------------------------------- what a mask hides, and other edges
@pytest.mark.parametrize("window", [0, 25])
@pytest.mark.parametrize("D,G,bits", [(128, 32, 4), (128, 16, 4), (256, 32, 8), (256, 32, 4)])
@pytest.mark.parametrize("q", [5, 90])
def test_attend_paged_masked_places_may_hold_anything(kvq, q, D, G, bits, window):
    """NaN and infinite scales reach the queries that attend their tokens, and no others (causal and
    window masks within the attended range, both kernels)."""
    kv = 150
    c = Cache(kvq, [kv, 40], [q, 1], 4, 1, D, G, bits, "srft", 16, seed=8, spoil=False)
    bad = {"k": (kv - 2, np.nan), "v": (kv - 3, np.nan), "vi": (kv - q + 1, np.inf)}
    for which, (t, val) in bad.items():
        page, off = c.table[0][t // 16], t % 16
        (c.ks if which == "k" else c.vs)[page, 0, off, 0] = val
    c.dev[1], c.dev[3] = torch.from_numpy(c.ks).cuda(), torch.from_numpy(c.vs).cuda()
    got = c.run(kvq, max_q_len=q, window=window).cpu().numpy().astype(np.float64)
    pos = np.arange(kv - q, kv)
    hit = np.zeros(q, bool)
    for t, _ in bad.values():
        hit |= (pos >= t) & ((pos - window < t) if window else True)
    assert hit.any() and not hit.all()
    assert np.isnan(got[:q][hit]).all()
    ok = ~np.concatenate([hit, [False]])
    with np.errstate(invalid="ignore", over="ignore"):
        ref = c.ref(window)
    check_rel_l2(got[ok].reshape(-1, D), ref[ok].reshape(-1, D), label="rows beside")


@pytest.mark.parametrize("Hq,Hkv,D", [(24, 2, 128), (40, 1, 128), (36, 1, 256), (5, 5, 128)])
def test_attend_paged_head_groups(kvq, Hq, Hkv, D):
    """Groups of query heads that do not fill, or do not fit, a tile of rows."""
    for q in ([1, 1], [3, 2], [50, 7]):
        c = Cache(kvq, [200, 77], q, Hq, Hkv, D, 32, 4, "srft", 32, seed=6)
        c.check(c.run(kvq, max_q_len=max(q)), label=f"q {q}")


def test_attend_paged_agrees_across_the_choice_of_kernel(kvq):
    """The same queries, told as longer than they are, go to the other kernel: the same formula."""
    c = Cache(kvq, [6000, 5800, 6100, 5900], [9, 8, 9, 9], 8, 2, 128, 32, 4, "srft", 16, seed=4)
    a = c.run(kvq, max_q_len=9).double()
    b = c.run(kvq, max_q_len=35).double()
    c.check(a)
    c.check(b)
    assert float((a - b).norm() / a.norm()) < 2e-3


def test_paged_calls_on_two_streams(kvq):
    """Calls with workspaces of their own may overlap."""
    cs = [Cache(kvq, [5000, 300], [1, 1], 8, 1, 128, 32, 4, "srft", 16, seed=1),
          Cache(kvq, [900, 700], [200, 300], 8, 2, 128, 32, 4, "srft", 16, seed=2)]
    want = [c.run(kvq, max_q_len=max(c.q_lens)) for c in cs]
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream(), torch.cuda.Stream()]
    ws = [kvq.make_paged_workspace(2, c.q.shape[1], c.kc.shape[1], 128, len(c.q), max(c.q_lens)) for c in cs]
    torch.cuda.synchronize()
    outs = [[torch.empty_like(w) for _ in range(6)] for w in want]
    for i in range(6):
        for c, s, w, o in zip(cs, ss, ws, outs):
            c.run(kvq, max_q_len=max(c.q_lens), workspace=w, out=o[i], stream=s)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, x) for x in o)


def test_paged_cache_past_32_bit_offsets(kvq):
    """Pages beyond 4 GB of codes: encode, decode and attention reach them."""
    D, H, P = 128, 8, 128
    plan, params = make_plan(kvq, D, "k")
    pages = (5 << 30) // (H * P * D // 2)
    codes = torch.empty((pages, H, P, D // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((pages, H, P, D // 32), dtype=torch.float16, device="cuda")
    vcodes, vscales = torch.empty_like(codes), torch.empty_like(scales)
    n = 300
    far = np.array([pages - 1, 0, pages - 2, pages // 2], np.int32)
    t = np.arange(n)
    slots = (far[t // P] * P + t % P).astype(np.int32)
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, n, H, D)).astype(np.float16)
    xd = torch.from_numpy(x).cuda()
    kvq.encode_paged([(plan, xd[0], codes, scales), (plan, xd[1], vcodes, vscales)], i32(slots))
    back = kvq.decode_paged(plan, codes, scales, i32(slots)).cpu().numpy().astype(np.float64)
    k = [a[torch.from_numpy(far).long().cuda()].cpu().numpy() for a in (codes, scales, vcodes, vscales)]
    near = np.arange(4, dtype=np.int32)
    nslots = (near[t // P] * P + t % P).astype(np.int32)
    check_rel_l2(back.reshape(-1, D), paged_ref.decoded(k[0], k[1], nslots, P, params, 32, "srft", 4).reshape(-1, D))
    for q in (1, 60):
        qs = rng.standard_normal((q, H, D)).astype(np.float16)
        got = kvq.attend_paged(plan, plan, torch.from_numpy(qs).cuda(), codes, scales, vcodes, vscales, i32(far[None]), i32([n]),
                               i32([0, q]), max_q_len=q).cpu().numpy().astype(np.float64)
        ref = paged_ref.attend(qs, *k, near[None], [n], [q], params, params, 32, "srft", 4)
        check_rel_l2(got.reshape(-1, D), ref.reshape(-1, D), label=f"q {q}")


def test_paged_cache_step_captured(kvq):
    """A whole serving step (plan, encode, attention) as a CUDA graph: replays go on from the state
    that the one before left, as eager steps do."""
    B, Hkv, Hq, D, P = 3, 2, 8, 128, 16
    made = []
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.standard_normal((2, B, Hkv, D)).astype(np.float16)).cuda()
    q = torch.from_numpy(rng.standard_normal((B, Hq, D)).astype(np.float16)).cuda()
    ones = torch.ones(B, dtype=torch.int32, device="cuda")
    for graph in (False, True):
        cache = kvq.PagedInt4KVCache(1, B, Hkv, D, 30, P, 6, kvgen.plan_params(D, seed=2, kind="k"), kvgen.plan_params(D, seed=2, kind="v"))
        out = torch.zeros_like(q)

        def step():
            s = cache.begin(ones, B)
            cache.update(0, x[0], x[1], s)
            cache.attend(0, q, s, max_q_len=1, out=out)
        step()
        torch.cuda.synchronize()
        if graph:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
        for _ in range(39):
            g.replay() if graph else step()
        torch.cuda.synchronize()
        assert cache.kv_lens.tolist() == [40] * B and int(cache.free_head.item()) == 9
        made.append((out, cache.block_table, cache.k_codes[0], cache.v_scales[0]))
    assert all(torch.equal(a, b) for a, b in zip(*made))


def test_paged_empty_calls(kvq):
    plan, _ = make_plan(kvq, 128, "k")
    z = torch.zeros
    kc, ks = z(2, 1, 16, 64, dtype=torch.uint8, device="cuda"), z(2, 1, 16, 4, dtype=torch.float16, device="cuda")
    assert kvq.decode_paged(plan, kc, ks, i32([])).shape == (0, 1, 128)
    kvq.encode_paged([(plan, z(0, 1, 128, dtype=torch.float16, device="cuda"), kc, ks)], i32([]))
    kvq.encode_paged([], i32([]))
    q = z(0, 4, 128, dtype=torch.float16, device="cuda")
    assert kvq.attend_paged(plan, plan, q, kc, ks, kc, ks, i32(np.zeros((0, 2))), i32([])).shape == (0, 4, 128)
    # requests without query tokens, and a request without pages
    q = torch.ones(1, 4, 128, dtype=torch.float16, device="cuda")
    out = kvq.attend_paged(plan, plan, q, kc, ks, kc, ks, i32([[0], [1], [1]]), i32([3, 0, 5]), i32([0, 0, 1, 1]), max_q_len=1)
    assert (out == 0).all()
    plan.close()
    with pytest.raises(ValueError, match="closed"):
        kvq.decode_paged(plan, kc, ks, i32([0]))
