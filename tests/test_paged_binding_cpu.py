"""The compiled binding of the paged calls: needed by them alone (no GPU)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT = """
import sys
sys.modules["rotated_int4_kv_b200._paged"] = None      # as if the file were not there
import rotated_int4_kv_b200 as kvq
assert kvq.Int4KVCache.compression_ratio(128, 32) > 3.5 and kvq.workspace_size(1, 8, 1, 128, 1024) > 0
assert kvq.paged_workspace_size(1, 8, 1, 128, 1, 1) > 0
for call in (lambda: kvq.page_plan(None, None, None, None, None, 16, 1), lambda: kvq.attend_paged(*[None] * 9)):
    try:
        call()
    except ImportError as e:
        assert "build.py" in str(e), e
    else:
        raise SystemExit("no error")
"""


def test_dense_calls_import_without_the_paged_binding():
    r = subprocess.run([sys.executable, "-c", WITHOUT], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
