"""Build libss2d.so (CUDA, sm_100a) in-tree with nvcc, and the Python module that marshals torch
tensors into the operators' calls with the host compiler.

Every .cu file under csrc/ is compiled to an object in _build/ (in parallel)
and linked into selective_scan_02_b200/libss2d.so with the CUDA runtime linked
statically, so the library depends only on the driver at run time.  The module
(csrc/marshal.cpp, selective_scan_02_b200/_marshal.so) is linked against it and against torch.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libss2d.so")
MARSHAL_SRC = os.path.join(CSRC, "marshal.cpp")
MARSHAL = os.path.join(PKG, "_marshal.so")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src, extra):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    if _stale(obj, [src] + _headers()):
        cmd = [NVCC, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if "--resource-usage" in extra or "-Xptxas=-v" in extra:
            sys.stderr.write(r.stderr)
    return obj


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile (if stale) and return the path of libss2d.so."""
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas=-v"] if verbose_ptxas else []
    srcs = _sources()
    if force:
        for o in glob.glob(os.path.join(BUILD, "*.o")):
            os.remove(o)
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra), srcs))
    if force or _stale(LIB, objs):
        cmd = [NVCC, *ARCH, "-shared", "-cudart", "static", "-Xlinker", "-soname=libss2d.so", "-o", LIB, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    build_marshal(force)
    return LIB


def build_marshal(force: bool = False) -> str:
    """Compile (if stale) and return the path of the marshalling module."""
    if not force and not _stale(MARSHAL, [MARSHAL_SRC, LIB] + _headers()):
        return MARSHAL
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    include = [sysconfig.get_paths()["include"], INCLUDE, os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"),
               *cpp_extension.include_paths()]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-I{d}" for d in include], MARSHAL_SRC,
           "-o", MARSHAL, LIB, "-Wl,-rpath,$ORIGIN", *[f"-L{d}" for d in cpp_extension.library_paths()],
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"building the marshalling module failed:\n{r.stdout}\n{r.stderr}")
    return MARSHAL


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
