"""Step planning where lengths and their sums pass 32 bits (exact, against the loop form)."""
import numpy as np
import pytest

from tests import paged_ref
from tests.test_gpu_paged import i32, kvq, no_device_errors  # noqa: F401  (fixtures)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TOP = 2 ** 31 - 1


@pytest.mark.parametrize("B,n", [(4, 50), (300, 50), (300, 9000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_requests_behind_sums_past_32_bits_are_served_in_full(kvq, B, n, in_place):  # noqa: F811
    """Refused requests of 2^31 - 1 tokens push the starts past 32 bits; those behind them still get
    their lengths, pages and table entries, and the slots that fit the map."""
    P, M, head = 16, 6, 3
    rng = np.random.default_rng(B)
    kv, q = rng.integers(0, 2 * P, B), rng.integers(0, 2 * P, B)
    q[1] = TOP
    q[B // 2 + 1] = TOP
    kv[B // 2 + 1] = 2
    q[2], kv[2] = 1, 5                      # fits its page
    q[3], kv[3] = 30, 20                    # needs pages
    table = rng.integers(0, 900, (B, M)).astype(np.int32)
    free = rng.permutation(5 * B + 9).astype(np.int32)
    # the loop form, with the refused requests' tokens left out of the map that it builds
    short = np.where(q == TOP, 0, q)
    ref = paged_ref.plan_step(kv, short, table, free, head, P, int(short.sum()))
    starts = np.minimum(np.concatenate([[0], np.cumsum(q.astype(np.int64))]), TOP)
    lens, h = i32(kv), i32([head])
    tab = i32(table)
    out = kvq.PagePlan.empty(B, n, "cuda")
    if in_place:
        out = out._replace(kv_lens=lens)
    kvq.page_plan(lens, i32(q), tab, i32(free), h, P, out=out)
    want_kv = np.where(q == TOP, kv, ref["kv_lens"])
    assert np.array_equal(out.kv_lens.cpu().numpy(), want_kv)
    assert np.array_equal(tab.cpu().numpy(), ref["table"])
    assert int(h.item()) == ref["head"]
    assert np.array_equal(out.q_starts.cpu().numpy(), starts)
    assert out.info.tolist() == [TOP, ref["info"][1], int((q == TOP).sum()), ref["info"][3]]
    # the map: request 0, then the refused request 1 to its end
    first = int(q[0])
    assert np.array_equal(out.slots.cpu().numpy()[:first], ref["slots"][:first])
    assert (out.slots[first:] == -1).all()
    assert np.array_equal(out.positions.cpu().numpy(), np.concatenate([kv[0] + np.arange(first), kv[1] + np.arange(n - first)]))


def test_a_request_whose_length_passes_32_bits_is_refused(kvq):  # noqa: F811
    """A table wide enough for more than 2^31 - 1 tokens of one request."""
    P, M = 128, 2 ** 24 + 4
    table = torch.zeros((1, M), dtype=torch.int32, device="cuda")
    free = i32(np.arange(10))
    for kv, q, served in ((TOP - 5, 5, True), (TOP - 5, 6, False), (TOP, 0, True), (TOP - 200, 201, False)):
        head = i32([0])
        step = kvq.page_plan(i32([kv]), i32([q]), table, free, head, P, q)
        assert step.kv_lens.tolist() == [kv + q if served else kv]
        assert step.info.tolist()[2] == (0 if served else 1)
        assert served or (int(head.item()) == 0 and (step.slots == -1).all())
        # positions past 2^31 - 1 saturate
        assert step.positions.tolist() == [min(kv + j, TOP) for j in range(q)]
