"""Paged attention where its two kernels (few query rows, prompts) differ in how they hold
numbers: V scales on both sides of the prompt kernel's limit, scales that are not finite, weights
far below a row's largest. Against the 64-bit form; tolerances as derived in tests/paged_ref.py."""
import numpy as np
import pytest

from tests.parity import rel_l2
from tests.test_gpu_paged import Cache, kvq, no_device_errors  # noqa: F401  (fixtures)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


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
