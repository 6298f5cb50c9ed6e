"""Builds libttq.so (the C-ABI library of the TTQ hot path) in-tree with nvcc for
sm_100a, and where torch is installed ``_host.so`` (the Python module that passes torch
tensors to its paged entry points) with the host compiler. Usage:
``python -m online_activation_aware_b200.build`` (or call ``build()``).

Object files go to ``_build/`` at the repository root; the shared libraries are written
next to this file so that the snapshot of the repository carries them."""

from __future__ import annotations

import importlib.util
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
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libttq.so")
HOST_SRC = os.path.join(CSRC, "host_binding.cpp")
HOST = os.path.join(PKG, "_host.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the TTQ library needs the CUDA toolkit to build")
    return cand


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps_mtime():
    paths = sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    paths.append(os.path.join(INCLUDE, "ttq.h"))
    return max(os.path.getmtime(p) for p in paths)


def build_host(verbose: bool = False, force: bool = False) -> str:
    """Compiles the Python module of the paged entry points against the installed torch."""
    import torch

    stamp = os.path.join(BUILD, "host.torch")
    built_for = open(stamp).read() if os.path.exists(stamp) else None
    newest = max(os.path.getmtime(HOST_SRC), os.path.getmtime(os.path.join(INCLUDE, "ttq.h")))
    if not force and built_for == torch.__version__ and os.path.exists(HOST) and os.path.getmtime(HOST) >= newest:
        return HOST
    os.makedirs(BUILD, exist_ok=True)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    torch_dir = os.path.dirname(torch.__file__)
    dirs = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(cuda, "include"),
            os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include")]
    tmp = HOST + ".tmp"
    cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-shared",
           f"-DTTQ_TORCH_VERSION=\"{torch.__version__}\"", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *(f"-I{d}" for d in dirs), HOST_SRC, "-o", tmp, "-L" + os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd))
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"the host compiler failed on {HOST_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, HOST)
    with open(stamp, "w") as f:
        f.write(torch.__version__)
    return HOST


def build(verbose: bool = False, force: bool = False, extra_flags=()) -> str:
    """Compiles every .cu under csrc/ and links libttq.so, then the host module beside it (where torch
    is installed: the C library needs nvcc only). Returns the library path."""
    if force or not os.path.exists(LIB) or os.path.getmtime(LIB) < _deps_mtime():
        build_library(verbose, extra_flags)
    if importlib.util.find_spec("torch") is not None:
        build_host(verbose, force)
    return LIB


def build_library(verbose: bool = False, extra_flags=()) -> None:
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd))
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    build(verbose="-v" in sys.argv, force="-f" in sys.argv)
    print(LIB)
