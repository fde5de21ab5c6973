"""The compiled binding of the paged calls: needed by them alone, and rebuilt when torch changes (no GPU)."""
import importlib.util
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


def test_binding_is_rebuilt_for_another_torch(tmp_path, monkeypatch):
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(ROOT, "rotated_int4_kv_b200", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "BINDING_LIB", str(tmp_path / "_paged.so"))
    monkeypatch.setattr(build, "_torch_version", lambda: "1.0")
    for version, builds in (("1.0", 1), ("1.0", 1), ("2.0", 2), ("2.0", 2), ("1.0", 3)):
        monkeypatch.setattr(build, "_torch_version", lambda: version)
        build._build_binding(False)
        assert len(ran) == builds, version
