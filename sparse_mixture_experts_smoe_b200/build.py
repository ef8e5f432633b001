"""Build libsmoe.so in-tree with nvcc for sm_100a, and the Python module beside it.

Each ``csrc/*.cu`` compiles to an object under ``_build/`` (in parallel, only
when its source or a header changed), then nvcc links the shared library next to
this file.  ``csrc/binding.cpp`` (torch tensors to the C entry points) compiles with
g++ into ``_binding.so``, which loads the library from its own folder.  Usage: ``python -m sparse_mixture_experts_smoe_b200.build [--force]``.
"""
from __future__ import annotations

import concurrent.futures as cf
import fcntl
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libsmoe.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_STAMP = os.path.join(BUILD, "binding.txt")  # what _binding.so was built for

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: cannot build libsmoe.so")


def _headers_mtime() -> float:
    hs = glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    return max(os.path.getmtime(h) for h in hs) if hs else 0.0


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    if (not os.path.exists(obj) or os.path.getmtime(obj) < os.path.getmtime(src)
            or os.path.getmtime(obj) < _headers_mtime()):
        cmd = [nvcc()] + ARCH + FLAGS + ["-c", src, "-o", obj + ".tmp"]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        subprocess.run(cmd, check=True)
        os.replace(obj + ".tmp", obj)
    return obj


def _binding_for() -> str:
    """What the built module depends on beside its sources: torch and the interpreter."""
    import torch
    return f"torch {torch.__version__}, {sys.implementation.cache_tag}"


def binding_stale() -> bool:
    """No module, or one built for another torch or Python (it would fail to load)."""
    if not os.path.exists(BINDING):
        return True
    if not os.path.exists(BINDING_STAMP):  # a package without its build folder: taken as it is
        return False
    with open(BINDING_STAMP) as f:
        return f.read() != _binding_for()


def _build_binding(force: bool) -> None:
    inputs = (BINDING_SRC, os.path.join(INCLUDE, "smoe.h"))
    if not force and not binding_stale() and os.path.exists(BINDING_STAMP) and \
            os.path.getmtime(BINDING) >= max(os.path.getmtime(p) for p in inputs):
        return
    import sysconfig

    import torch
    cuda, home = os.path.dirname(os.path.dirname(nvcc())), os.path.dirname(torch.__file__)
    dirs = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(cuda, "include"),
            os.path.join(home, "include"), os.path.join(home, "include/torch/csrc/api/include")]
    lib = os.path.join(home, "lib")
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += [f"-I{d}" for d in dirs] + [BINDING_SRC, "-o", tmp, f"-L{PKG}", "-lsmoe", "-Wl,-rpath,$ORIGIN",
                                       f"-L{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
                                       "-ltorch_python"]
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    with open(BINDING_STAMP, "w") as f:
        f.write(_binding_for())


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with open(os.path.join(BUILD, ".lock"), "w") as lock:
        fcntl.flock(lock, fcntl.LOCK_EX)
        if force:
            for o in glob.glob(os.path.join(BUILD, "*.o")):
                os.remove(o)
        srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
        with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
            objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
        newest = max(os.path.getmtime(o) for o in objs)
        if force or not os.path.exists(LIB) or os.path.getmtime(LIB) < newest:
            tmp = LIB + ".tmp"
            subprocess.run([nvcc()] + ARCH + ["-shared", "-o", tmp] + objs, check=True)
            os.replace(tmp, LIB)
        _build_binding(force)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
