"""Builds libsparge.so (the C-ABI CUDA library, for sm_100a) and the extension module
_serving (the argument checks of serving.py's calls, host C++) in-tree.

    python -m free_block_sparse_predict_b200.build

Each .cu file under csrc/ is compiled to an object in _build/ (in parallel),
then linked into free_block_sparse_predict_b200/libsparge.so.  Objects are
rebuilt when their source or any header is newer.  _serving carries the
interpreter's tag in its name and is rebuilt for another torch too.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libsparge.so")
BINDING = os.path.join(PKG, "_serving" + sysconfig.get_config_var("EXT_SUFFIX"))
STAMP = os.path.join(BUILD, "serving.torch")  # the torch that BINDING was built for

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libsparge")


def _headers():
    return glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    newest_dep = max([os.path.getmtime(src)] + [os.path.getmtime(h) for h in _headers()])
    if os.path.exists(obj) and os.path.getmtime(obj) >= newest_dep:
        return obj
    cmd = [nvcc(), "-c", src, "-o", obj, "-I", INCLUDE] + ARCH + FLAGS + list(extra)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def _torch_version() -> str:
    return importlib.metadata.version("torch")


def _binding_is_current(src: str) -> bool:
    newest = max(os.path.getmtime(src), os.path.getmtime(os.path.join(INCLUDE, "sparge.h")))
    if not os.path.exists(BINDING) or os.path.getmtime(BINDING) < newest:
        return False
    if not os.path.exists(STAMP):
        return False
    with open(STAMP) as f:
        return f.read() == _torch_version()


def _binding() -> None:
    src = os.path.join(CSRC, "serving_binding.cpp")
    if _binding_is_current(src):
        return
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    inc = os.path.join(torch, "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    dirs = [INCLUDE, inc, os.path.join(inc, "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"], cuda]
    cmd = ["g++", "-shared", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f'-DSPARGE_TORCH_VERSION="{_torch_version()}"', src, "-o", BINDING]
    cmd += [x for d in dirs for x in ("-isystem" if d != INCLUDE else "-I", d)]
    cmd += ["-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {src}:\n{r.stdout}\n{r.stderr}")
    with open(STAMP, "w") as f:
        f.write(_torch_version())


def build(extra=(), verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    with cf.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        binding = ex.submit(_binding)
        objs = list(ex.map(lambda s: _compile(s, extra), srcs))
    newest = max(os.path.getmtime(o) for o in objs)
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < newest:
        cmd = [nvcc(), "-shared", "-o", LIB] + objs + ARCH
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    binding.result()  # behind the C library, which knows nothing of torch
    if verbose:
        print(LIB)
    return LIB


if __name__ == "__main__":
    build(extra=sys.argv[1:], verbose=True)
