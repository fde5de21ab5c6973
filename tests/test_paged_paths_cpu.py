"""The choice between the two paged attention kernels, on the host (no GPU needed)."""
import pytest

pytest.importorskip("torch")


def test_attend_paged_path_setting():
    import rotated_int4_kv_b200 as kvq

    lib = kvq.lib
    assert kvq.get_attend_paged_path() == "auto"
    assert lib.kvq_set_attend_paged_path(3) == -1 and lib.kvq_set_attend_paged_path(-1) == -1
    assert kvq.get_attend_paged_path() == "auto"
    with pytest.raises(KeyError):
        kvq.set_attend_paged_path("tensor")
    size = kvq.paged_workspace_size
    auto = size(64, 32, 8, 128, 64, 64)
    try:
        kvq.set_attend_paged_path("few")
        assert kvq.get_attend_paged_path() == "few"
        few = size(64, 32, 8, 128, 64, 64)
        # at most n_q Gq / 8 + B row tiles of 8.8 KB per head, whatever the bound; 64 with it at 1
        assert size(64, 32, 8, 128, 64, 1) < few <= size(64, 32, 8, 128, 64, 1) + 32 * 8 * 9000
        kvq.set_attend_paged_path("prompt")
        assert size(64, 32, 8, 128, 64, 64) == size(1, 8, 8, 256, 1, 1) > 0
    finally:
        kvq.set_attend_paged_path("auto")
    assert size(64, 32, 8, 128, 64, 64) == auto
