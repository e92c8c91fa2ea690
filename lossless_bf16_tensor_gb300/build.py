"""Build liblct.so (the C-ABI library) for sm_103a with nvcc, and _calls.so (the
Python entry points of its gradient and adapter calls) with the C++ compiler,
in-tree.

Each translation unit is compiled in parallel, then linked into one shared
library beside this file.  The results are rebuilt only when a source or header
is newer than them.  No GPU is needed to build.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "liblct.so")
CALLS_SRC = os.path.join(HERE, "calls", "calls.cpp")
CALLS = os.path.join(HERE, "_calls.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2,-ffp-contract=off",
              "-Xptxas", "-warn-spills", "-I" + INCLUDE]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build liblct")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _deps() -> list[str]:
    return sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def is_stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in _deps())


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and not is_stale():
        return LIB
    nvcc = _nvcc()
    tmpdir = tempfile.mkdtemp(prefix="lct_build_", dir=HERE)
    try:
        def compile_one(src: str) -> str:
            obj = os.path.join(tmpdir, os.path.basename(src) + ".o")
            cmd = [nvcc] + ARCH + NVCC_FLAGS + ["-c", src, "-o", obj]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError("nvcc failed on %s:\n%s%s" % (src, r.stdout, r.stderr))
            if verbose and (r.stdout or r.stderr):
                print(r.stdout + r.stderr)
            return obj

        with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
            objs = list(ex.map(compile_one, sources()))
        out = os.path.join(tmpdir, "liblct.so")
        cmd = [nvcc] + ARCH + ["-shared", "-o", out] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
        os.replace(out, LIB)
    finally:
        shutil.rmtree(tmpdir, ignore_errors=True)
    return LIB


def build_calls(force: bool = False) -> str:
    """_calls.so, linked against liblct.so beside it and the installed torch."""
    deps = [CALLS_SRC, LIB, os.path.abspath(__file__)] + glob.glob(os.path.join(INCLUDE, "*.h"))
    if not force and os.path.exists(CALLS) and all(os.path.getmtime(p) <= os.path.getmtime(CALLS) for p in deps):
        return CALLS
    import torch
    root = os.path.join(os.path.dirname(torch.__file__))
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_path("include"), os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")]
    tmpdir = tempfile.mkdtemp(prefix="lct_build_", dir=HERE)
    try:
        out = os.path.join(tmpdir, "_calls.so")
        cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", CALLS_SRC, "-o", out,
               "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI)]
        cmd += ["-I" + p for p in include] + ["-L" + os.path.join(root, "lib"), "-L" + HERE]
        cmd += ["-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-l:liblct.so", "-Wl,-rpath,$ORIGIN"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("building _calls.so failed:\n%s%s" % (r.stdout, r.stderr))
        os.replace(out, CALLS)
    finally:
        shutil.rmtree(tmpdir, ignore_errors=True)
    return CALLS


if __name__ == "__main__":  # pragma: no cover
    import sys
    print(build_library(force="--force" in sys.argv, verbose=True))
    print(build_calls(force="--force" in sys.argv))
