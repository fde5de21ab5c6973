"""Both kernels of the paged attention (few query rows, prompts), each chosen by the setting and
run over the whole range: head_dim 128 and 256, masks, windows, empty rows, bad pages, far pages,
captured calls, and V scales on both sides of the prompt kernel's limit. Against the 64-bit form;
tolerances as derived in tests/paged_ref.py."""
import numpy as np
import pytest

import kvgen
import oracle
from tests import paged_ref
from tests.parity import check_rel_l2, rel_l2
from tests.test_gpu_paged import Cache, i32, kvq, make_plan, no_device_errors  # noqa: F401  (fixtures)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(params=["few", "prompt"])
def path(kvq, request):  # noqa: F811
    kvq.set_attend_paged_path(request.param)
    yield request.param
    kvq.set_attend_paged_path("auto")


FORMS = [(32, 4, "srft"), (16, 4, "srht"), (32, 8, "srht"), (16, 8, "srft")]
HEADS = [(12, 2, 128), (32, 8, 128), (8, 1, 128), (4, 1, 256), (3, 3, 128), (2, 2, 256), (40, 1, 128), (36, 1, 256)]


def put_scales(c):
    c.dev[1], c.dev[3] = torch.from_numpy(c.ks).cuda(), torch.from_numpy(c.vs).cuda()


def scale_tokens(c, b, which, tokens, factor):
    """Multiply the K or V scales of request b's tokens."""
    s = c.ks if which == "k" else c.vs
    t = np.asarray(tokens)
    at = (c.table[b][t // c.P], slice(None), t % c.P)
    s[at] = np.minimum(s[at].astype(np.float64) * factor, 65504).astype(np.float16)


def check_rows(c, got, window=0, tol=2e-3, label=""):
    """Row by row; rows whose value leaves fp16 are not compared."""
    ref = c.ref(window)
    got = got.detach().cpu().numpy()[: len(ref)].astype(np.float64)
    ok = (np.abs(ref) < 6e4).all(-1)
    assert ok.mean() > 0.5, label
    r = rel_l2(got[ok], ref[ok])
    assert r.max() <= tol, f"{label}: rel L2 worst row {r.max():.3e} (tol {tol})"


# sizes at which the prompt kernel is the one chosen
PROMPTS = {128: dict(kv=[2048], q=[256], Hq=8, Hkv=1), 256: dict(kv=[4096], q=[300], Hq=4, Hkv=1)}


@pytest.mark.parametrize("window", [0, 150])
@pytest.mark.parametrize("big", ["front", "middle", "back", "one", "alternate"])
@pytest.mark.parametrize("D,G,bits", [(128, 32, 4), (128, 16, 8), (256, 32, 4), (256, 16, 8)])
def test_prompt_attention_with_v_scales_across_the_limit(kvq, D, G, bits, big, window):
    """V scales from 2^12 (8 bits: 2^9) on are held divided by a power of two: tiles with such
    scales before, after and between tiles without."""
    s = PROMPTS[D]
    c = Cache(kvq, s["kv"], s["q"], s["Hq"], s["Hkv"], D, G, bits, "srft", 64, seed=11, spoil=False)
    n, m = s["kv"][0], s["q"][0]
    # scales are (0.5 .. 1.5) / Qmax: of size 20 (2) everywhere, from 4200 (520) on where they are large
    scale_tokens(c, 0, "v", np.arange(n), 20 * 7 if bits == 4 else 2 * 127)
    # within what the queries attend with a window too
    spots = {"front": np.arange(0, n - m), "middle": np.arange(n - m + 20, n - m + 60), "back": np.arange(n - 40, n),
             "one": np.array([n - m + 33]), "alternate": np.arange(0, n, 256)}
    scale_tokens(c, 0, "v", spots[big], 420.0 if bits == 4 else 520.0)
    put_scales(c)
    check_rows(c, c.run(kvq, max_q_len=m, window=window), window, label=f"{big} window {window}")


# ---------------------------------------------------------------- each kernel over the whole range
@pytest.mark.parametrize("G,bits,xf", FORMS)
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_each_kernel_over_lengths_and_masks(kvq, path, Hq, Hkv, D, G, bits, xf):
    """Single tokens, several, prompts; tiles, pages and row blocks that end inside; requests without
    tokens, without queries, with more queries than tokens."""
    for seed, (P, kv, q, w) in enumerate((
            (16, [1, 17, 300, 0], [1, 1, 1, 1], 0), (64, [63, 64, 65, 700, 2], [1, 1, 1, 1, 1], 40),
            (32, [300, 9, 40], [7, 0, 6], 33), (16, [3, 50], [6, 2], 0), (128, [129, 257], [70, 1], 0),
            (64, [330, 70, 128], [130, 33, 128], 0), (16, [400, 5], [65, 5], 100))):
        c = Cache(kvq, kv, q, Hq, Hkv, D, G, bits, xf, P, seed=seed, pad=3)
        out = torch.full((sum(q) + 3, Hq, D), 5.0, dtype=torch.float16, device="cuda")
        c.check(c.run(kvq, max_q_len=max(q), window=w, out=out), window=w, label=f"kv {kv} q {q} window {w}")
        assert (out[sum(q):] == 5.0).all()   # rows of no request stay


@pytest.mark.parametrize("D,G,bits", [(128, 32, 4), (256, 32, 4), (256, 16, 8)])
def test_each_kernel_on_long_caches(kvq, path, D, G, bits):
    """Units cut into pieces that several CTAs share; many of them, and row blocks of several units."""
    for kv, q, P, w in (([9000, 3, 500], [1, 1, 1], 64, 0), ([5000, 4097], [1, 5], 16, 300), ([3000], [300], 32, 0),
                        ([2500, 40, 2300], [90, 40, 150], 128, 700)):
        c = Cache(kvq, kv, q, 4, 1, D, G, bits, "srft", P, seed=21)
        c.check(c.run(kvq, max_q_len=max(q), window=w), window=w, label=f"kv {kv} q {q}")


@pytest.mark.parametrize("B", [300, 1300])
def test_each_kernel_with_many_requests(kvq, path, B):
    rng = np.random.default_rng(B)
    kv, q = rng.integers(0, 40, B), rng.integers(0, 3, B)
    for q in (q, np.where(rng.random(B) < 0.05, 30, q)):
        c = Cache(kvq, kv, q, 4, 1, 128, 32, 4, "srft", 16, seed=3)
        c.check(c.run(kvq, max_q_len=int(q.max())))


@pytest.mark.parametrize("window", [0, 25])
@pytest.mark.parametrize("D,G,bits", [(128, 32, 4), (128, 16, 4), (128, 32, 8), (256, 32, 8), (256, 16, 8), (256, 32, 4)])
@pytest.mark.parametrize("q", [5, 90])
def test_each_kernel_keeps_masked_places_apart(kvq, path, q, D, G, bits, window):
    """NaN scales reach the queries that attend their tokens, and no others, also within a tile."""
    kv = 150
    c = Cache(kvq, [kv, 40], [q, 1], 4, 1, D, G, bits, "srft", 16, seed=8, spoil=False)
    bad = {"k": kv - 2, "v": kv - q + 1}
    for which, t in bad.items():
        (c.ks if which == "k" else c.vs)[c.table[0][t // 16], 0, t % 16, -1] = np.nan
    put_scales(c)
    got = c.run(kvq, max_q_len=q, window=window).cpu().numpy().astype(np.float64)
    pos = np.arange(kv - q, kv)
    hit = np.zeros(q, bool)
    for t in bad.values():
        hit |= (pos >= t) & ((pos - window < t) if window else True)
    assert hit.any() and not hit.all()
    assert np.isnan(got[:q][hit]).all()
    ok = ~np.concatenate([hit, [False]])
    with np.errstate(invalid="ignore", over="ignore"):
        ref = c.ref(window)
    check_rel_l2(got[ok].reshape(-1, D), ref[ok].reshape(-1, D), label="rows beside")


@pytest.mark.parametrize("D,bits", [(128, 4), (128, 8), (256, 4), (256, 8)])
@pytest.mark.parametrize("q", [1, 90])
def test_each_kernel_over_the_range_of_scales(kvq, path, q, D, bits):
    """V and K scales over fp16's whole range, all alike and with large ones in some tokens only."""
    for vs, ks in ((9000.0, 1.0), (6e-7, 1.0), (1.0, 3e4), (300.0, 40.0)):
        for where in (slice(0, 300), slice(0, 60), slice(130, 150)):
            c = Cache(kvq, [300], [q], 4, 1, D, 32, bits, "srft", 16, seed=5, q_size=1.0 / ks)
            for which, by in (("k", ks), ("v", vs)):
                scale_tokens(c, 0, which, np.arange(300)[where], by * (7 if which == "v" and by > 1 else 1))
            put_scales(c)
            ref = c.ref()
            got = c.run(kvq, max_q_len=q).cpu().numpy()
            fits = np.abs(ref) < 6e4
            big = np.where(fits, ref, 0)
            # fp16 outputs: half a step is at least 2^-25, whatever the value
            err = np.abs(np.where(fits, got, 0) - big)
            assert (err <= 4e-3 * np.abs(big).max(-1, keepdims=True) + 2.0 ** -24).all(), (vs, ks, where)


@pytest.mark.parametrize("window", [0, 60])
@pytest.mark.parametrize("big", ["front", "middle", "one", "alternate"])
@pytest.mark.parametrize("D,G,bits", [(128, 32, 4), (256, 32, 8)])
def test_each_kernel_with_v_scales_across_the_limit(kvq, path, D, G, bits, big, window):
    """As above, at sizes where one unit holds rows that attend the large tokens and rows that do not."""
    n, m = 700, 120
    c = Cache(kvq, [n], [m], 2, 1, D, G, bits, "srft", 32, seed=12, spoil=False)
    scale_tokens(c, 0, "v", np.arange(n), 20 * 7 if bits == 4 else 2 * 127)
    spots = {"front": np.arange(0, n - m + 5), "middle": np.arange(n - m + 20, n - m + 40), "one": np.array([n - m - 20]),
             "alternate": np.arange(0, n, 150)}
    scale_tokens(c, 0, "v", spots[big], 420.0 if bits == 4 else 520.0)
    put_scales(c)
    check_rows(c, c.run(kvq, max_q_len=m, window=window), window, label=f"{big} window {window}")


def test_each_kernel_raises_a_flag_for_bad_pages(kvq, path):
    for D in (128, 256):
        c = Cache(kvq, [400], [30], 4, 1, D, 32, 4, "srft", 16, spoil=False)
        for bad in (-1, 10 ** 6):
            c.tab[0, 3] = bad
            got = c.run(kvq, max_q_len=30)
            torch.cuda.synchronize()
            assert kvq.poll_device_errors() == 8 and torch.isfinite(got).all()
        c = Cache(kvq, [500], [100], 4, 1, D, 32, 4, "srft", 16)
        c.tab[0, :20] = -1                       # no attended token lies there
        c.check(c.run(kvq, max_q_len=100, window=40), window=40)
        # no pages at all: nothing to attend to
        q = torch.ones(9, 4, D, dtype=torch.float16, device="cuda")
        out = kvq.attend_paged(c.pk, c.pv, q, *c.dev, torch.empty((1, 0), dtype=torch.int32, device="cuda"), i32([9]), i32([0, 9]))
        assert (out == 0).all()


@pytest.mark.parametrize("D", [128, 256])
def test_each_kernel_is_deterministic_and_captures(kvq, path, D):
    for q in ([1, 1, 1], [40, 1, 25]):
        c = Cache(kvq, [3000, 41, 777], q, 12, 2, D, 32, 4, "srft", 16)
        want = c.run(kvq, max_q_len=max(q))
        ws = kvq.make_paged_workspace(3, 12, 2, D, sum(q), max(q))
        out = torch.zeros_like(want)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        c.run(kvq, max_q_len=max(q), workspace=ws, out=out, stream=side)
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
        c.kv[0] = 1500                           # new lengths in place: the captured call follows them
        c.lens[0] = 1500
        g.replay()
        c.check(out)


def test_each_kernel_cuts_lengths_to_the_bounds(kvq, path):
    c = Cache(kvq, [100, 40], [6, 2], 4, 1, 128, 32, 4, "srft", 16)
    out, full = (torch.full((8, 4, 128), 5.0, dtype=torch.float16, device="cuda") for _ in range(2))
    c.run(kvq, max_q_len=4, out=out)
    c.run(kvq, max_q_len=6, out=full)
    assert (out[4:6] == 5.0).all()
    assert rel_l2(out[:4].double().cpu(), full[:4].double().cpu()).max() < 2e-3
    c.lens = i32([250, 40])       # past the table's (7 + 1) pages of 16: cut to max_kv_len
    c.check(c.run(kvq, max_q_len=6, max_kv_len=100))


def test_kernels_agree(kvq):
    """The same queries through both: the same formula, other roundings."""
    for D, G, bits in ((128, 32, 4), (128, 16, 8), (256, 32, 4), (256, 16, 8)):
        c = Cache(kvq, [6000, 580, 61], [9, 80, 2], 8, 2, D, G, bits, "srft", 16, seed=4)
        got = []
        try:
            for path in ("few", "prompt"):
                kvq.set_attend_paged_path(path)
                got.append(c.run(kvq, max_q_len=80).double())
        finally:
            kvq.set_attend_paged_path("auto")
        c.check(got[0])
        c.check(got[1])
        assert not torch.equal(*got)


def test_each_kernel_past_32_bit_offsets(kvq, path):
    """Pages beyond 4 GB of codes."""
    H, P = 8, 128
    for D, bits in ((128, 4), (256, 8)):
        plan, params = make_plan(kvq, D, "k", bits=bits)
        row = D * bits // 8
        pages = (9 << 29) // (H * P * row)
        far = np.array([pages - 1, 0, pages - 2, pages // 2], np.int32)
        rng = np.random.default_rng(1)
        c = Cache(kvq, [300], [1], H, H, D, 32, bits, "srft", P, seed=3, spoil=False)   # random pages to place far away
        big = []
        for a in c.dev:
            t = torch.empty((pages, *a.shape[1:]), dtype=a.dtype, device="cuda")
            t[torch.from_numpy(far).long().cuda()] = a[:4]
            big.append(t)
        near = [a[:4].cpu().numpy() for a in c.dev]
        for q in (1, 60):
            qs = rng.standard_normal((q, H, D)).astype(np.float16)
            got = kvq.attend_paged(plan, plan, torch.from_numpy(qs).cuda(), *big, i32(far[None]), i32([300]), i32([0, q]), max_q_len=q)
            ref = paged_ref.attend(qs, *near, np.arange(4, dtype=np.int32)[None], [300], [q], params, params, 32, "srft", bits)
            check_rel_l2(got.cpu().numpy().astype(np.float64).reshape(-1, D), ref.reshape(-1, D), label=f"q {q}")
        del big


@pytest.mark.parametrize("D", [128, 256])
def test_cache_class_through_each_kernel(kvq, path, D):
    """A prompt, then single tokens, through the class; the attention checked on what the pages hold."""
    B, Hkv, Hq, P, n = 2, 2, 8, 32, 90
    kp, vp = kvgen.plan_params(D, seed=2, kind="k"), kvgen.plan_params(D, seed=2, kind="v")
    cache = kvq.PagedInt4KVCache(1, B, Hkv, D, 12, P, 6, kp, vp)
    rng = np.random.default_rng(5)
    length = [0, 0]
    for q in ([n, 40], [1, 1], [0, 3]):
        t = sum(q)
        step = cache.begin(i32(q), t)
        x = torch.from_numpy(rng.standard_normal((2, t, Hkv, D)).astype(np.float16)).cuda()
        cache.update(0, x[0], x[1], step)
        qs = rng.standard_normal((t, Hq, D)).astype(np.float16)
        got = cache.attend(0, torch.from_numpy(qs).cuda(), step, max_q_len=max(q)).cpu().numpy().astype(np.float64)
        length = [a + b for a, b in zip(length, q)]
        pages = [a[0].cpu().numpy() for a in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]
        want = paged_ref.attend(qs, *pages, cache.block_table.cpu().numpy(), length, q, kp, vp, 32, "srft", 4)
        check_rel_l2(got.reshape(-1, D), want.reshape(-1, D), label=f"{q}")


# ---------------------------------------------------------------- scales that are not finite
@pytest.mark.parametrize("bad", [np.inf, -np.inf])
@pytest.mark.parametrize("D,G,bits", [(128, 32, 4), (128, 16, 8), (256, 32, 4), (256, 16, 4), (256, 32, 8)])
@pytest.mark.parametrize("q", [3, 90])
def test_each_kernel_makes_infinite_k_scales_nan(kvq, path, q, D, G, bits, bad):
    """An infinite K scale would give the score -inf, as masked places have, where its group's sum is
    negative: the queries that attend its token get NaN all the same, and no others."""
    kv, window = 200, 50
    for t in (kv - 2, kv - q - 20, kv - q - 60):       # attended by the last queries, by all or the first, by none
        c = Cache(kvq, [kv, 40], [q, 1], 8, 2, D, G, bits, "srft", 16, seed=9, spoil=False)
        c.ks[c.table[0][t // 16], :, t % 16, -1] = bad
        put_scales(c)
        got = c.run(kvq, max_q_len=q, window=window).cpu().numpy().astype(np.float64)
        pos = np.arange(kv - q, kv)
        hit = np.concatenate([(pos >= t) & (pos - window < t), [False]])
        assert hit.any() == (t != kv - q - 60)
        assert np.isnan(got[hit]).all()
        with np.errstate(invalid="ignore", over="ignore"):
            ref = c.ref(window)
        check_rel_l2(got[~hit].reshape(-1, D), ref[~hit].reshape(-1, D), label="rows beside")


@pytest.mark.parametrize("D,bits", [(128, 4), (256, 8)])
@pytest.mark.parametrize("q", [2, 90])
def test_each_kernel_sees_a_score_of_minus_infinity(kvq, path, q, D, bits):
    """A group of equal codes under an infinite scale, and queries whose rotated form is -1 there and 0
    elsewhere: every product is -inf or 0 and the token's score exactly that of a masked place."""
    kv = 150
    c = Cache(kvq, [kv], [q], 1, 1, D, 32, bits, "srft", 16, seed=10, spoil=False)
    signs, lam = (np.asarray(a, np.float64) for a in c.kp)
    basis = np.asarray(oracle.srft_forward(np.eye(D), signs, np.ones(D), "srft"), np.float64)   # [sample, channel]
    c.q[:] = (basis[:, :32] @ -lam[:32]).astype(np.float16)
    c.qd.copy_(torch.from_numpy(c.q).cuda())
    t = kv - 1
    page = c.table[0][t // 16]
    c.kc[page, 0, t % 16, : 32 * bits // 8] = 0x11 if bits == 4 else 1
    c.ks[page, 0, t % 16, 0] = np.inf
    c.dev[0] = torch.from_numpy(c.kc).cuda()
    put_scales(c)
    got = c.run(kvq, max_q_len=q).cpu().numpy()
    assert np.isnan(got[-1]).all() and np.isfinite(got[:-1]).all()


@pytest.mark.parametrize("D,G,bits", [(128, 32, 4), (128, 16, 4), (256, 32, 8), (256, 16, 4)])
def test_a_scale_that_is_no_number_leaves_its_tile_as_precise(kvq, path, D, G, bits):
    """Tokens with small scales beside one with a NaN: the queries that do not attend that one are as
    near the formula as without it."""
    kv, window, t = 130, 30, 20
    for which, size in (("v", 5e-4), ("k", 2e-3)):
        c = Cache(kvq, [kv], [100], 2, 1, D, G, bits, "srft", 16, seed=13, spoil=False, q_size=1.0 if which == "v" else 2.0 ** -3 / size)
        scale_tokens(c, 0, which, np.arange(kv), size)
        (c.ks if which == "k" else c.vs)[c.table[0][t // 16], 0, t % 16, 1] = np.nan
        put_scales(c)
        got = c.run(kvq, max_q_len=100, window=window).cpu().numpy().astype(np.float64)
        with np.errstate(invalid="ignore"):
            ref = c.ref(window)
        ok = np.arange(kv - 100, kv) - window >= t
        # fp16 outputs of this size are subnormal: half a step, 2^-25, per element beside the usual 2e-3
        err = np.linalg.norm((got - ref)[ok], axis=-1)
        assert (err <= 2e-3 * np.linalg.norm(ref[ok], axis=-1) + 2.0 ** -25 * np.sqrt(D)).all(), which


# ---------------------------------------------------------------- weights far below the largest
@pytest.mark.parametrize("D,G,bits", [(128, 32, 4), (128, 16, 8), (256, 32, 4), (256, 32, 8)])
@pytest.mark.parametrize("vsize", [0.1, 10.0, 30000.0])
@pytest.mark.parametrize("sink", ["first", "last"])
@pytest.mark.parametrize("q", [1, 40])
def test_each_kernel_weighs_a_tail_below_a_sink(kvq, path, q, sink, vsize, D, G, bits):
    """One token whose score is 8 to 17.5 above that of thousands, and whose V is 0: the output is the tail's
    alone, its weights 2^-11 to 2^-25 of the largest. Queries along the sink's K, so that its score has no
    cancelling terms, and V of one sign, so that lost weights do not average out."""
    n = 4000
    for gap in (8.0, 13.3, 16.0, 17.5):
        if gap > 16 and vsize > 1:
            continue      # weights below 2^-24 times 30000 are beyond what the few-row kernel's range holds
        c = Cache(kvq, [n], [q], 1, 1, D, G, bits, "srft", 64, seed=15, spoil=False)
        t0 = 0 if sink == "first" else n - q
        at = (c.table[0][t0 // 64], slice(None), t0 % 64)
        scale_tokens(c, 0, "k", np.arange(n), 0.0)
        c.ks[at] = 1.0 if bits == 4 else 1.0 / 16
        signs, lam = (np.asarray(a, np.float64) for a in c.kp)
        slot = np.array([c.table[0][t0 // 64] * 64 + t0 % 64])
        y = oracle.srft_forward(paged_ref.decoded(c.kc, c.ks, slot, 64, c.kp, *c.form)[0, 0], signs, lam, "srft")
        aim = oracle.srft_inverse(lam ** 2 * y, signs, lam, "srft")          # R^T lambda y: q~ = y
        c.q[:] = (aim * gap * np.sqrt(D) / (y @ y)).astype(np.float16)
        c.qd.copy_(torch.from_numpy(c.q).cuda())
        codes = np.abs(oracle.unpack_codes(c.vc, bits)).astype(np.int8)
        c.vc = oracle.pack_codes(codes, bits).view(np.uint8).reshape(c.vc.shape)
        c.dev[2] = torch.from_numpy(c.vc).cuda()
        scale_tokens(c, 0, "v", np.arange(n), vsize * (7 if bits == 4 else 127))
        c.vs[at] = 0.0
        put_scales(c)
        ref = c.ref()
        if np.abs(ref).max() > 6e4:
            continue      # the outputs leave fp16
        # Everything else 2e-3 (tests/paged_ref.py); the score's relative error, sqrt(3) roundings of rms
        # 2^-11 / sqrt(3) averaged over D like terms, times the score, three standard deviations; and the
        # kernels' bounds on a weight, relative to the largest: 2^-32 (prompt); 2^-37 for the weight and again, of a
        # scale of 1, for its product with the scale, both 2^16 larger for scales from 2^15 on.
        tail = np.exp(gap)
        tol = 2e-3 + 3 * 2.0 ** -11 * gap / np.sqrt(D)
        tol += tail * (2.0 ** -32 if path == "prompt" else 2.0 ** -37 * (1 + 2 / vsize) if vsize < 1 else 2.0 ** (-37 + np.log2(vsize) + 2))
        got = c.run(kvq, max_q_len=q).cpu().numpy().astype(np.float64)
        check_rel_l2(got.reshape(-1, D), ref.reshape(-1, D), tol=tol, label=f"gap {gap}")


def test_cache_class_workspaces_stay_within_twice_the_largest(kvq):
    """Steps that grow a little each time: the workspaces kept for captured graphs add up to no more
    than the one in use."""
    B, Hkv, Hq, D = 64, 1, 8, 256
    params = kvgen.plan_params(D, seed=2, kind="k")
    cache = kvq.PagedInt4KVCache(1, B, Hkv, D, 70, 16, 2, params, params)
    kvq.set_attend_paged_path("few")                       # its workspace grows with the bounds
    try:
        for n in range(8, 200, 8):
            step = cache.begin(i32([1] * B), B)
            q = torch.ones((n, Hq, D), dtype=torch.float16, device="cuda")
            cache.attend(0, q, step, max_q_len=n)
            cache.kv_lens.zero_()
            cache.free_head.zero_()
        torch.cuda.synchronize()
        need = kvq.paged_workspace_size(B, Hq, Hkv, D, n, n)
    finally:
        kvq.set_attend_paged_path("auto")
    now = cache._ws[Hq].numel()
    kept = sum(w.numel() for w in cache._grown)
    assert need <= now <= 2 * need and kept <= now


# ---------------------------------------------------------------- factors
@pytest.mark.parametrize("D,G,bits,xf", [(128, 32, 4, "srft"), (128, 16, 8, "srht"), (256, 32, 4, "srht"), (256, 16, 8, "srft")])
@pytest.mark.parametrize("q", [1, 70])
def test_each_kernel_with_factors_of_seven_decades(kvq, path, q, D, G, bits, xf):
    """Factors from 3e-4 to 3e3, a group of channels each, and scales in proportion, as an encode would
    give: every channel counts alike in the scores and in the output."""
    n = 300
    c = Cache(kvq, [n, 40], [q, 2], 4, 1, D, G, bits, xf, 32, seed=16, spoil=False)
    lam = np.repeat(np.random.default_rng(1).permutation(np.logspace(-3.5, 3.5, D // G)), G)
    for which in "kv":
        signs = kvgen.plan_params(D, seed=17, kind=which)[0]
        params = (signs, lam.astype(np.float32))
        plan = kvq.Plan(*params, G, xf, bits)
        s = c.ks if which == "k" else c.vs
        s[:] = (s.astype(np.float64) * lam[::G]).astype(np.float16)
        if which == "k":
            c.pk, c.kp = plan, params
        else:
            c.pv, c.vp = plan, params
    # scales of 3e-4 / 127 keep 2 to 7 bits in fp16: the reference reads the same ones
    put_scales(c)
    c.check(c.run(kvq, max_q_len=max(q, 2)))


def test_plans_hold_no_matrices_for_paged_calls(kvq):
    """What plans hold on the device: the codec's own operands (2 D^2 halves to encode, D^2 to decode) and
    4 KB, the rest shared."""
    D, n = 256, 64
    first = make_plan(kvq, D, "k")[0]
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    plans = [make_plan(kvq, D, "k", seed=s)[0] for s in range(n)]
    used = before - torch.cuda.mem_get_info()[0]
    own = 3 * D * D * 2 + 4096
    # the allocator hands out 2 MB blocks
    assert used <= n * own * 1.4 + (4 << 20), used / n
    del first, plans


# ---------------------------------------------------------------- loose bounds
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (5, 1, 128), (24, 2, 128), (4, 1, 256)])
@pytest.mark.parametrize("B", [1, 3, 40, 70, 1100])
def test_bounds_need_not_be_tight(kvq, path, B, Hq, Hkv, D):
    """Without max_q_len (so n, as if one request had every token): single tokens, idle requests, a
    longer one among them, padding; the same values as with the tight bound."""
    rng = np.random.default_rng(B)
    kv = rng.integers(1, 60, B)
    for q in (np.ones(B, int), rng.integers(0, 3, B), np.where(rng.random(B) < 0.1, 37, rng.integers(0, 2, B))):
        q[rng.integers(B)] = 1
        c = Cache(kvq, kv, q, Hq, Hkv, D, 32, 4, "srft", 16, seed=B, pad=2)
        out = torch.full((int(q.sum()) + 2, Hq, D), 5.0, dtype=torch.float16, device="cuda")
        c.run(kvq, out=out)
        assert (out[q.sum():] == 5.0).all()
        tight = c.run(kvq, max_q_len=int(q.max()))[: q.sum()]
        assert torch.equal(out[: q.sum()], tight) or rel_l2(out[: q.sum()].double().cpu(), tight.double().cpu()).max() < 2e-3
        if B < 1000:
            c.check(out)


def test_a_loose_bound_keeps_the_workspace_and_the_kernel(kvq):
    """A decode batch whose longest query is not told: the workspace is that of its tokens, and the few-row
    kernel takes it (bit for bit the values that it gives)."""
    B, Hq, Hkv = 64, 32, 8
    need = kvq.paged_workspace_size(B, Hq, Hkv, 128, B, B)
    kvq.set_attend_paged_path("few")
    try:
        few = kvq.paged_workspace_size(B, Hq, Hkv, 128, B, B)
        assert few < 1.2 * kvq.paged_workspace_size(B, Hq, Hkv, 128, B, 1) + (4 << 20)
        c = Cache(kvq, [300] * B, [1] * B, Hq, Hkv, 128, 32, 4, "srft", 64, seed=2, spoil=False)
        want = c.run(kvq)
    finally:
        kvq.set_attend_paged_path("auto")
    assert few <= need
    assert torch.equal(c.run(kvq), want)


# ---------------------------------------------------------------- calls that follow one another closely
@pytest.mark.parametrize("q_hi", [1, 40])
def test_steps_in_a_row_read_what_the_call_before_wrote(kvq, path, q_hi):
    """Release, planning, encode and attention start early, while the call in front still runs: many steps
    without a wait on the host leave the same state and outputs as steps that wait after every call."""
    B, Hkv, Hq, D, P, M = 24, 2, 8, 128, 16, 12
    params = kvgen.plan_params(D, seed=2, kind="k"), kvgen.plan_params(D, seed=2, kind="v")
    made = []
    for wait in (True, False):
        rng = np.random.default_rng(9)
        cache = kvq.PagedInt4KVCache(1, B, Hkv, D, 200, P, M, *params)
        steps, outs = [], []
        for _ in range(60):
            q = rng.integers(0, q_hi + 1, B)
            n = B * q_hi
            x = torch.from_numpy(rng.standard_normal((2, n, Hkv, D)).astype(np.float16)).cuda()
            qs = torch.from_numpy(rng.standard_normal((n, Hq, D)).astype(np.float16)).cuda()
            steps.append((i32(q), torch.from_numpy(rng.random(B) < 0.15).cuda(), x, qs, torch.zeros((n, Hq, D), dtype=torch.float16, device="cuda")))
        sync = torch.cuda.synchronize if wait else (lambda: None)
        torch.cuda.synchronize()
        for q, done, x, qs, out in steps:
            step = cache.begin(q, x.shape[1])
            sync()
            cache.update(0, x[0], x[1], step)
            sync()
            outs.append(cache.attend(0, qs, step, max_q_len=q_hi, out=out))
            sync()
            outs.append(kvq.decode_paged(cache.k_plans[0], cache.k_codes[0], cache.k_scales[0], step.slots))
            sync()
            cache.release(done)
            sync()
        torch.cuda.synchronize()
        made.append((*outs, cache.kv_lens, cache.free_head, cache.free_pages, cache.block_table, cache.k_codes[0], cache.v_scales[0]))
    assert all(torch.equal(a, b) for a, b in zip(*made))


@pytest.mark.parametrize("D,G,bits,n", [(128, 32, 4, 40), (256, 16, 8, 40), (256, 16, 4, 700), (128, 32, 8, 3000)])
def test_decode_reads_what_the_encode_before_wrote(kvq, D, G, bits, n):
    """The same slots encoded and decoded over and over without a wait: every decode gives the rows of
    the encode in front of it, none of the one before."""
    plan, _ = make_plan(kvq, D, "k", G=G, bits=bits)
    pages = n // 16 + 2
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    xs = torch.randn(2, n, 1, D, generator=g, device="cuda").half()
    slots = torch.randperm(pages * 16, generator=g, device="cuda")[:n].int()
    codes = torch.zeros((pages, 1, 16, D * bits // 8), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((pages, 1, 16, D // G), dtype=torch.float16, device="cuda")
    want = []
    for x in xs:
        kvq.encode_paged([(plan, x, codes, scales)], slots)
        torch.cuda.synchronize()
        want.append(kvq.decode_paged(plan, codes, scales, slots))
        torch.cuda.synchronize()
    outs = [torch.empty_like(want[0]) for _ in range(100)]
    for i, out in enumerate(outs):
        kvq.encode_paged([(plan, xs[i % 2], codes, scales)], slots)
        kvq.decode_paged(plan, codes, scales, slots, out=out)
    torch.cuda.synchronize()
    assert all(torch.equal(out, want[i % 2]) for i, out in enumerate(outs))
