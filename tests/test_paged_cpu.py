"""The paged entry points on the host: refusals before any CUDA call, workspace sizes, and the
plain form of the step planner against a hand-worked example (no GPU needed)."""
import ctypes

import numpy as np
import pytest

from tests import paged_ref

torch = pytest.importorskip("torch")
P, F0 = ctypes.c_void_p, ctypes.c_float(0)
ONE = (ctypes.c_int32 * 64)()


def _buf():
    return ctypes.cast(ONE, P)


def test_page_plan_refusals():
    from rotated_int4_kv_b200 import lib

    def call(B=1, M=1, stride=1, n_free=1, page=16, n_slots=1, kv=_buf(), head=_buf(), info=_buf()):
        x = _buf()
        return lib.kvq_page_plan(kv, x, B, x, M, stride, x, n_free, head, x, page, x, x, n_slots, x, x, info, None)

    assert call(B=-1) == -1 and call(M=2, stride=1) == -1 and call(n_free=-1) == -1 and call(n_slots=-1) == -1
    assert call(page=8) == -2 and call(page=48) == -2 and call(page=256) == -2 and call(page=0) == -2
    assert call(B=16385) == -2
    assert call(kv=None) == -1 and call(head=None) == -1 and call(info=None) == -1
    assert b"null" in lib.kvq_last_error()
    x = _buf()
    assert lib.kvq_page_release(x, x, x, 0, 1, 1, 16, x, 1, x, None) == -1
    assert lib.kvq_page_release(x, x, x, 1, 1, 1, 12, x, 1, x, None) == -2
    assert lib.kvq_page_release(None, x, x, 1, 1, 1, 16, x, 1, x, None) == -1
    assert lib.kvq_page_release(None, None, None, 0, 0, 0, 16, None, 0, None, None) == 0


def test_paged_codec_refusals():
    from rotated_int4_kv_b200 import _lib, lib

    jobs = (_lib.PagedEncodeJob * 1)()
    x = _buf()
    assert lib.kvq_encode_paged(jobs, 1, 4, 1, 16, 1, x, None) == -1          # null plan
    assert b"job 0" in lib.kvq_last_error()
    assert lib.kvq_encode_paged(None, 1, 4, 1, 16, 1, x, None) == -1
    assert lib.kvq_encode_paged(jobs, 1, -1, 1, 16, 1, x, None) == -1
    assert lib.kvq_encode_paged(jobs, 1, 4, 1, 24, 1, x, None) == -2          # page size
    assert lib.kvq_encode_paged(jobs, 1, 4, 129, 16, 1, x, None) == -2        # heads
    assert lib.kvq_encode_paged(jobs, 1, 4, 0, 16, 1, x, None) == -1
    assert lib.kvq_encode_paged(jobs, 1, 4, 1, 16, 0, x, None) == -1
    assert lib.kvq_encode_paged(jobs, 1, 4, 1, 128, 1 << 24, x, None) == -2   # slots past 32 bits
    assert lib.kvq_encode_paged(jobs, 0, 4, 1, 16, 1, x, None) == 0
    assert lib.kvq_decode_paged(None, x, x, 1, 16, 1, x, 1, x, None) == -1


def test_attend_paged_refusals():
    from rotated_int4_kv_b200 import lib

    x = _buf()
    assert lib.kvq_attend_paged(None, None, x, 128, 128, x, x, x, x, 1, 16, x, 1, 1, x, None, 1, 1, 1, 1, 1, 16, 0, F0,
                                x, x, 1 << 30, None) == -1
    assert b"null plan" in lib.kvq_last_error()


def test_workspace_sizes():
    import rotated_int4_kv_b200 as kvq

    size = kvq.paged_workspace_size
    assert size(0, 8, 1, 128, 1, 1) == 0 and size(1, 7, 2, 128, 1, 1) == 0 and size(1, 8, 1, 96, 1, 1) == 0
    assert size(1, 8, 1, 128, -1, 1) == 0 and size(1, 8, 1, 128, 1, 0) == 0
    prev = 0
    for n in (1, 8, 100, 1000):
        s = size(4, 32, 8, 128, n, n)
        assert s >= prev and s % 16 == 0
        prev = s
    assert size(64, 32, 8, 128, 64, 1) >= size(1, 32, 8, 128, 1, 1)


def test_wrappers_refuse_host_tensors_and_bad_shapes():
    import rotated_int4_kv_b200 as kvq

    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        kvq.page_plan(i32, i32, torch.zeros(2, 3, dtype=torch.int32), i32, i32[:1], 16, 4)
    with pytest.raises(ValueError, match="CUDA"):
        kvq.page_release(torch.zeros(2, dtype=torch.bool), i32, torch.zeros(2, 3, dtype=torch.int32), i32, i32[:1], 16)
    with pytest.raises((ValueError, TypeError)):
        kvq.page_plan([1], [1], None, None, None, 16, 4)
    with pytest.raises((ValueError, TypeError)):
        kvq.attend_paged(None, None, torch.zeros(2, 8, 128), None, None, None, None, i32, i32)


def test_plain_plan_by_hand():
    # page size 16: request 0 (15 + 3) needs one page, 1 is idle, 2 (fresh, 17) needs two, 3 fits its page,
    # 4 wants more pages than its row holds; four free entries from the head on
    table = np.array([[7, -1, -1], [3, -1, -1], [-1, -1, -1], [9, -1, -1], [1, 2, 4]], np.int32)
    r = paged_ref.plan_step([15, 5, 0, 3, 40], [3, 0, 17, 1, 20], table, np.array([50, 51, 52, 53, 54], np.int32), 1, 16, 44)
    assert r["table"][0].tolist() == [7, 51, -1] and r["table"][2].tolist() == [52, 53, -1]
    assert r["slots"][:3].tolist() == [7 * 16 + 15, 51 * 16, 51 * 16 + 1]
    assert r["slots"][3:20].tolist() == [52 * 16 + i for i in range(16)] + [53 * 16]
    assert r["slots"][20] == 9 * 16 + 3 and r["slots"][21:41].tolist() == [-1] * 20
    assert r["positions"][21:].tolist() == list(range(40, 60)) + [-1] * 3
    assert r["kv_lens"].tolist() == [18, 5, 17, 4, 40] and r["head"] == 4
    assert r["info"].tolist() == [41, 3, 1, 3] and r["q_starts"].tolist() == [0, 3, 3, 20, 21, 41]
