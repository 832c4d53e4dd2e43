"""Build libpa.so (planner + sm_100a kernels + C ABI) and _cache_ops.so (the
session-cache operators on torch tensors, over libpa.so) in the package directory.

nvcc compiles every CUDA source for sm_100a only (-gencode
arch=compute_100a,code=sm_100a) with -lineinfo; the host planner is C++17.
cudart is linked statically so the library does not depend on the runtime
version another package in the process brings.
"""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
REPO = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(REPO, "include")
BUILD = os.path.join(REPO, "_build")
LIB = os.path.join(HERE, "libpa.so")
TORCH_OPS = os.path.join(HERE, "_cache_ops.so")
STAMP = os.path.join(BUILD, "_cache_ops.made_for")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
CU_SOURCES = ["kernels.cu", "capi.cu", "noalloc.cu", "rope_append.cu", "window_attend.cu", "weigh.cu", "evict.cu"]
CPP_SOURCES = ["plan.cpp"]
HEADERS = ["plan.h", "ptx.cuh", "sessions.cuh", "tmap.h", "umma.cuh"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpa.so")


def _newer(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _read(path: str) -> str:
    if not os.path.exists(path):
        return ""
    with open(path) as f:
        return f.read()


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(INCLUDE, "pa.h")]
    objs = []
    cc = nvcc()
    common = ["-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]
    for src in CU_SOURCES + CPP_SOURCES:
        path = os.path.join(CSRC, src)
        obj = os.path.join(BUILD, src + ".o")
        objs.append(obj)
        if force or _newer(obj, [path] + headers):
            if src.endswith(".cu"):
                cmd = [cc] + ARCH + common + ["-lineinfo", "-Xptxas", "-v" if verbose else "-O3", "-c", path, "-o", obj]
            else:
                cmd = ["g++", "-O3", "-std=c++17", "-fPIC", "-Wall", "-I", INCLUDE, "-I", CSRC,
                       "-I", "/usr/local/cuda/include", "-c", path, "-o", obj]
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            subprocess.check_call(cmd)
    if force or _newer(LIB, objs):
        tmp = LIB + ".tmp"
        subprocess.check_call([cc] + ARCH + ["-shared", "-o", tmp] + objs)
        os.replace(tmp, LIB)
    build_torch_ops(force, verbose)
    return LIB


def build_torch_ops(force: bool = False, verbose: bool = False):
    """The Python module _cache_ops (csrc/torch_ops.cpp), against the installed
    torch; libpa.so is found beside it ($ORIGIN).  Without torch or its headers it is
    left out (None), with a line on stderr: the C ABI and the planned path need
    neither.  Built anew for another torch or Python than it was built for."""
    try:
        version = importlib.metadata.version("torch")
        root = os.path.dirname(importlib.util.find_spec("torch").origin)
    except (importlib.metadata.PackageNotFoundError, AttributeError):
        root = None
    if root is None or not os.path.isdir(os.path.join(root, "include", "torch")):
        print("torch or its headers are not installed: _cache_ops.so (the session-cache operators on torch tensors) "
              "is not built", file=sys.stderr)
        return None
    made_for = f"torch {version} python {sys.version}"
    src = os.path.join(CSRC, "torch_ops.cpp")
    os.makedirs(BUILD, exist_ok=True)
    if not (force or _newer(TORCH_OPS, [src, os.path.join(INCLUDE, "pa.h")]) or _read(STAMP) != made_for):
        return TORCH_OPS
    import sysconfig

    import torch
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    tmp = TORCH_OPS + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={abi}",
           "-I", INCLUDE, "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", "/usr/local/cuda/include", "-isystem", sysconfig.get_paths()["include"], src, "-o", tmp,
           "-L", HERE, "-lpa", "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
           "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(tmp, TORCH_OPS)
    with open(STAMP, "w") as f:
        f.write(made_for)
    return TORCH_OPS


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
