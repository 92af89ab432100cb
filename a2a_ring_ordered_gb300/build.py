"""Build ``lib/libccl.so`` in-tree with nvcc for sm_103a (GB300), and the
binding's ``lib/_tensors.so`` with g++ against the installed torch (where there
is one).

Each translation unit compiles in parallel, then one link step produces the
shared library (CUDA runtime linked statically, so the library needs only the
driver at run time).  Rebuilds only when a source or header is newer than the
library.  Usage: ``python -m a2a_ring_ordered_gb300.build [--force] [-v]``.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libccl.so")
TENSORS = os.path.join(LIBDIR, "_tensors.so")
TENSORS_SRC = os.path.join(CSRC, "tensors.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = [
    "-O3", "-lineinfo", "-std=c++17", "-DNDEBUG",
    "-Xcompiler", "-fPIC,-O2,-Wall",
    "-I", INCLUDE, "-I", CSRC,
]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libccl.so")
    return cand


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps() -> list[str]:
    return sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) \
        + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def _newer(product: str, deps: list[str]) -> bool:
    if not os.path.exists(product):
        return False
    t = os.path.getmtime(product)
    return all(os.path.getmtime(d) <= t for d in deps)


def up_to_date() -> bool:
    return _newer(LIB, _deps())


def _torch() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        raise RuntimeError("torch is required to build _tensors.so")
    return list(spec.submodule_search_locations)[0]


def build_tensors(force: bool = False, verbose: bool = False) -> str:
    """Compile the binding's helper if needed; returns its path."""
    torch = _torch()
    if not force and _newer(TENSORS, [TENSORS_SRC, os.path.abspath(__file__), os.path.join(torch, "version.py")]):
        return TENSORS
    os.makedirs(LIBDIR, exist_ok=True)
    include = os.path.join(torch, "include")
    tmp = TENSORS + ".tmp"
    gxx = shutil.which("g++")
    if gxx is None:
        raise RuntimeError("g++ is required to build _tensors.so")
    cmd = [gxx, "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall", "-o", tmp, TENSORS_SRC,
           "-isystem", include, "-isystem", os.path.join(include, "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        if os.path.exists(TENSORS):  # of another source or another torch
            os.remove(TENSORS)
        raise RuntimeError(f"g++ failed on tensors.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, TENSORS)
    return TENSORS


def _compile(src: str, verbose: bool, ptxas_v: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
    if ptxas_v:
        cmd += ["-Xptxas", "-v"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    if ptxas_v or verbose:
        sys.stdout.write(r.stdout + r.stderr)
    return obj


def build(force: bool = False, verbose: bool = False, ptxas_v: bool = False) -> str:
    """Compile and link the library, and the binding's helper, if needed;
    returns the library's path.  The C ABI needs no torch, nor does the binding
    need its helper: where that cannot be built, a warning says why."""
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        helper = ex.submit(build_tensors, force, verbose)
        lib = _build_library(force, verbose, ptxas_v)
        try:
            helper.result()
        except RuntimeError as e:
            warnings.warn(f"the binding's helper was not built: {e}", RuntimeWarning, stacklevel=2)
    return lib


def _build_library(force: bool, verbose: bool, ptxas_v: bool) -> str:
    if not force and not ptxas_v and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose, ptxas_v), srcs))
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "--cudart", "static", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    ap.add_argument("--ptxas-v", action="store_true", help="print registers / spills per kernel")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose, ptxas_v=a.ptxas_v))


if __name__ == "__main__":
    main()
