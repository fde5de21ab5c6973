"""Build the in-tree shared library ``libkvq.so`` (CUDA C++ for sm_100a) with nvcc, and the Python
extension ``_paged.so`` over its paged calls with g++.

Usage: ``python rotated_int4_kv_b200/build.py [--force] [--verbose]`` (run it as a script:
importing the package loads the library it builds). Object files
go to ``_build/`` at the repository root; the library is written next to this file.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import importlib.metadata
import os
import shutil
import subprocess
import sysconfig
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libkvq.so")
SOURCES = ["kvq_api.cu", "kvq_codec.cu", "kvq_encode_tc.cu", "kvq_decode_tc.cu", "kvq_attend.cu",
           "kvq_plan_basis.cu", "kvq_page_plan.cu", "kvq_attend_paged.cu", "kvq_attend_prompt.cu"]
BINDING = "paged_binding.cpp"   # the Python extension module _paged (torch's C++ interface, linked to libkvq.so)
BINDING_LIB = os.path.join(PKG, "_paged.so")
HEADERS = ["kvq_internal.h", "kvq_ptx.cuh", "kvq_quant.cuh", "srft_fft.cuh"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-v", "-I" + os.path.join(ROOT, "include")]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "kvq.h")]
    objs, jobs = [], []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + hdrs):
            jobs.append((s, o))

    def run(job):
        s, o = job
        cmd = [nvcc, *ARCH, *FLAGS, "-c", s, "-o", o]
        r = subprocess.run(cmd, capture_output=True, text=True)
        log = o.replace(".o", ".log")
        with open(log, "w") as f:
            f.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {os.path.basename(s)}:\n{r.stderr[-4000:]}")
        return log

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 1))) as ex:
        for log in ex.map(run, jobs):
            if verbose:
                print(open(log).read())
    if force or jobs or _stale(LIB, objs):
        cmd = [nvcc, *ARCH, "-shared", "-Xlinker", "-soname=libkvq.so", "-o", LIB, *objs, "-lrt"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n" + r.stderr[-4000:])
    _build_binding(force)
    return LIB


def _torch_version() -> str:
    return importlib.metadata.version("torch")


def _build_binding(force: bool) -> None:
    """Rebuilt for a changed source, header or library, and for another torch or Python than its stamp names."""
    src = os.path.join(CSRC, BINDING)
    stamp, made_for = os.path.join(BUILD, "paged_binding.stamp"), f"torch {_torch_version()} python {sys.version}"
    same = os.path.exists(stamp) and open(stamp).read() == made_for
    if not force and same and not _stale(BINDING_LIB, [src, os.path.join(ROOT, "include", "kvq.h"), LIB]):
        return
    import torch
    t = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{d}" for d in (os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
                                os.path.join(cuda, "include"), sysconfig.get_paths()["include"])),
           src, "-o", BINDING_LIB, LIB, f"-L{os.path.join(t, 'lib')}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda",
           "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{os.path.join(t, 'lib')}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    with open(os.path.join(BUILD, "paged_binding.log"), "w") as f:
        f.write(r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {BINDING}:\n{r.stderr[-4000:]}")
    with open(stamp, "w") as f:
        f.write(made_for)


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose=a.verbose))
    return 0


if __name__ == "__main__":
    sys.exit(main())
