"""Build the decoder's shared library in-tree with nvcc for sm_100a.

``python -m kv_cache_decode_dualcache_b200.build`` (or ``build()``) compiles
``csrc/*.cu`` into ``libfdllm.so`` next to this file, and the Python binding of
the stream-ordered operators into ``_binding.so`` (a warning where torch's
headers or g++ do not allow it; the library does not need it).  Nothing is
JIT-compiled at import time; the binding loads the prebuilt library and fails
loudly when it is missing.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libfdllm.so")
# Self-checking variant: every device access of the GEMM / epilogue bounds-
# checked, violations recorded and reported as FDLLM_ERR_CUDA.
LIB_CHECKS = os.path.join(HERE, "libfdllm_checks.so")
# Python binding of the stream-ordered operators (an extension module over
# torch's C++ interface; host code only).
BINDING = os.path.join(HERE, "_binding.so")
BINDING_STAMP = os.path.join(ROOT, "_build", "binding.stamp")   # what it was built for
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfdllm.so")


def sources():
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.cu")))


def _inputs():
    return sources() + sorted(glob.glob(os.path.join(HERE, "csrc", "*.cuh"))) + sorted(
        glob.glob(os.path.join(HERE, "csrc", "*.h"))) + [os.path.join(ROOT, "include", "fdllm.h")]


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in _inputs())


def build_binding(force: bool = False, verbose: bool = False) -> str:
    import sysconfig

    src = os.path.join(HERE, "csrc", "binding.cpp")
    import torch

    inputs = (src, os.path.join(ROOT, "include", "fdllm.h"))
    stamp = f"python {sys.version} torch {torch.__version__} {os.path.dirname(torch.__file__)}"
    if not force and os.path.exists(BINDING) and os.path.exists(BINDING_STAMP) and all(
            os.path.getmtime(p) <= os.path.getmtime(BINDING) for p in inputs):
        with open(BINDING_STAMP) as f:
            if f.read() == stamp:
                return BINDING
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-shared", "-fPIC", "-O2", "-std=c++17", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), src, "-o", tmp, "-L", os.path.join(root, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda",
           "-Wl,-rpath," + os.path.join(root, "lib")]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    try:
        r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        if r.returncode != 0:
            raise RuntimeError("g++ failed on binding.cpp:\n" + r.stdout.decode(errors="replace"))
    except (OSError, RuntimeError):
        if os.path.exists(BINDING):   # of another torch, or of older sources
            os.remove(BINDING)
        raise
    os.replace(tmp, BINDING)
    os.makedirs(os.path.dirname(BINDING_STAMP), exist_ok=True)
    with open(BINDING_STAMP, "w") as f:
        f.write(stamp)
    return BINDING


def build(force: bool = False, verbose: bool = False, extra=None, checks: bool = False) -> str:
    lib = build_library(LIB_CHECKS if checks else LIB, force, verbose, extra, checks)
    try:
        build_binding(force, verbose)
    except (ImportError, OSError, RuntimeError) as e:
        warnings.warn(f"the Python binding of the stream-ordered operators was not built: {e}", RuntimeWarning)
    return lib


def build_library(lib: str, force: bool, verbose: bool, extra, checks: bool) -> str:
    if not force and up_to_date(lib):
        return lib
    nvcc = _nvcc()
    objdir = os.path.join(ROOT, "_build", "checks" if checks else "release")
    os.makedirs(objdir, exist_ok=True)
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler",
                    "-fvisibility=hidden", "-I", os.path.join(ROOT, "include"),
                    "--expt-relaxed-constexpr"] + (["-DFDLLM_CHECKS"] if checks else []) + \
        list(extra or [])
    objs = []
    procs = []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [nvcc, "-c", src, "-o", obj] + flags
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT), src))
        objs.append(obj)
    for p, src in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{out.decode(errors='replace')}")
        if verbose and out:
            print(out.decode(errors="replace"), file=sys.stderr)
    tmp = lib + ".tmp"
    cmd = [nvcc, "-shared", "-o", tmp] + objs + ARCH + ["-Xcompiler", "-fPIC"]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout.decode(errors="replace"))
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                checks="--checks" in sys.argv))
