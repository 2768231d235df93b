"""Builds libhpc_decode.so in-tree with nvcc for sm_103a (GB300).

Each translation unit is compiled in parallel, then linked against the
shared CUDA runtime. The library is rebuilt when any source or header is
newer than it. Nothing here runs at import time of the package.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB_NAME = "libhpc_decode.so"
LIB_PATH = os.path.join(OUT_DIR, LIB_NAME)
# the Python binding's fast calls; left out where Python's headers are missing
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING_PATH = os.path.join(OUT_DIR, f"hpc_binding.{sys.implementation.cache_tag}.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libhpc_decode.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _python_include():
    path = sysconfig.get_path("include")
    return path if path and os.path.exists(os.path.join(path, "Python.h")) else None


def _headers():
    return glob.glob(os.path.join(INCLUDE, "*.h"))


def _inputs():
    return _sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        _headers() + [os.path.abspath(__file__)]


def _older(path, inputs) -> bool:
    """Whether the built file is missing or older than something it is made of."""
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(f) > t for f in inputs)


def binding_is_stale() -> bool:
    """The extension module calls the library by the descriptors and signatures it was compiled
    with: one older than them (another interpreter's, which rebuilt the library only) is not used."""
    return _older(BINDING_PATH, [BINDING_SRC, os.path.abspath(__file__)] + _headers())


def is_stale() -> bool:
    return _older(LIB_PATH, _inputs()) or (_python_include() is not None and binding_is_stale())


def common_flags():
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                   "-I", INCLUDE, "-I", CSRC]


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link what is stale; returns the library path."""
    if not force and not is_stale():
        return LIB_PATH
    os.makedirs(OUT_DIR, exist_ok=True)
    cc = nvcc()
    if force or _older(LIB_PATH, _inputs()):
        _build_library(cc, verbose, extra_flags)
    if _python_include() and (force or binding_is_stale()):
        tmp = BINDING_PATH + f".tmp{os.getpid()}"
        _run([cc, "-O2", "-std=c++17", "-shared", "-cudart", "none", "-Xcompiler", "-fPIC",
              "-I", INCLUDE, "-I", _python_include(), BINDING_SRC, "-o", tmp], f"nvcc failed on {BINDING_SRC}")
        os.replace(tmp, BINDING_PATH)
    return LIB_PATH


def _build_library(cc: str, verbose: bool, extra_flags):
    srcs = _sources()

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.basename(src) + ".o")
        cmd = [cc, *common_flags(), *extra_flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        said = _run(cmd, f"nvcc failed on {src}")
        if verbose and said:
            print(said, flush=True)
        return obj

    with ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    _run([cc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "shared"], "link failed")
    os.replace(tmp, LIB_PATH)


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
