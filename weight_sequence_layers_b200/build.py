"""Builds the in-tree CUDA library libttt.so for sm_100a with nvcc, and where torch is installed
_bind.so, the binding's argument checks, with the host compiler.

Each csrc/*.cu is compiled separately (in parallel) to an object, then linked into one
shared library with the CUDA runtime linked statically, so the library loads on a host
without a GPU driver (the driver entry point for tensor-map encoding is looked up at run
time). Usage: python -m weight_sequence_layers_b200.build [--force] [--verbose-ptxas]
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libttt.so")
BIND = os.path.join(PKG, "_bind.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include")]


def _deps():
    return sorted(glob.glob(os.path.join(CSRC, "*"))) + [os.path.join(ROOT, "include", "ttt.h")]


def _compile(src: str, ptxas_v: bool) -> str:
    obj = os.path.join(OBJ, os.path.basename(src) + ".o")
    cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
    if ptxas_v:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
    if ptxas_v:
        sys.stderr.write(r.stderr)
    return obj


def _bind_stamp(torch_dir: str) -> str:
    """What _bind.so was built against: it is built again where the interpreter or torch changes."""
    with open(os.path.join(torch_dir, "version.py")) as f:
        return f"{sys.version}\n{torch_dir}\n{f.read()}"


def _build_bind(force: bool = False) -> bool:
    """Builds _bind.so where torch and its headers are there; the binding works without it, and the
    library needs neither. Returns whether it is built and up to date."""
    src, stamp_file = os.path.join(CSRC, "bind.cpp"), os.path.join(OBJ, "bind.stamp")
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return False
    torch = spec.submodule_search_locations[0]
    try:
        stamp = _bind_stamp(torch)
    except OSError:
        return False
    old = open(stamp_file).read() if os.path.exists(stamp_file) else None
    if not force and old == stamp and os.path.exists(BIND) and \
            os.path.getmtime(BIND) >= os.path.getmtime(src):
        return True
    if os.path.exists(BIND):
        os.remove(BIND)  # one built against another torch must not be loaded
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC",
           "-I", os.path.join(torch, "include"), "-I", sysconfig.get_paths()["include"], src,
           "-o", BIND, "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        failed = r.stderr if r.returncode != 0 else None
    except OSError as e:  # no compiler
        failed = str(e)
    if failed is not None:
        sys.stderr.write(f"_bind.so is not built (its checks are then made in Python): {failed}\n")
        return False
    os.makedirs(OBJ, exist_ok=True)
    with open(stamp_file, "w") as f:
        f.write(stamp)
    return True


def build(force: bool = False, ptxas_v: bool = False) -> str:
    lib = _build_lib(force, ptxas_v)
    _build_bind(force)
    return lib


def _build_lib(force: bool, ptxas_v: bool) -> str:
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    newest = max(os.path.getmtime(p) for p in _deps())
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= newest:
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, ptxas_v), srcs))
    cmd = [NVCC, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-cudart", "static", *objs, "-o", LIB]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, ptxas_v="--verbose-ptxas" in sys.argv)
    print(LIB)
