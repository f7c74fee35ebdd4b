"""Builds the CUDA library libslikl.so in-tree with nvcc for sm_100a, and beside it, where torch is installed,
_slikl_torch.so, the C++ marshalling of torch tensors for the calls whose latency counts (g++, no device
code). The library alone needs neither torch nor Python's headers.

Usage: python -m sparse_lightning_indexer_b200.build [--force]
"""

from __future__ import annotations

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
LIB = os.path.join(PKG, "libslikl.so")
TORCH_LIB = os.path.join(PKG, "_slikl_torch.so")
OBJDIR = os.path.join(PKG, "_build")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-Xptxas", "-v",
    "-I", INCLUDE, "-I", CSRC,
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every csrc/*.cu into one shared library, and the torch binding where what it needs is
    there; returns the library's path."""
    os.makedirs(OBJDIR, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")))
    objs = []
    for src in sources:
        obj = os.path.join(OBJDIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            cmd = [_nvcc(), *NVCC_FLAGS, "-c", src, "-o", obj]
            res = subprocess.run(cmd, capture_output=True, text=True)
            log = os.path.join(OBJDIR, os.path.basename(src)[:-3] + ".ptxas.txt")
            with open(log, "w") as f:
                f.write(res.stdout + res.stderr)
            if res.returncode != 0:
                sys.stderr.write(res.stdout + res.stderr)
                raise RuntimeError(f"nvcc failed on {src}")
            if verbose:
                sys.stderr.write(res.stderr)
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [_nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp,
               *objs, "-lcuda"]
        subprocess.check_call(cmd)
        os.replace(tmp, LIB)
    missing = _binding_lacks()
    if missing:
        sys.stderr.write(f"_slikl_torch.so is not built: no {missing}\n")
    else:
        build_torch(force)
    return LIB


def _torch_root():
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _binding_lacks():
    """What the torch binding needs and is not installed, or None."""
    root = _torch_root()
    if not root:
        return "torch"
    for path in (os.path.join(root, "lib", "libc10_cuda.so"), os.path.join(root, "include", "ATen", "ATen.h"),
                 os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        if not os.path.exists(path):
            return path
    return None if shutil.which("g++") else "g++"


def build_torch(force: bool = False) -> str:
    """Compile csrc/slikl_torch.cpp against torch's headers and libslikl.so; returns its path. A module
    built for another torch or Python than the installed ones is built anew."""
    src = os.path.join(CSRC, "slikl_torch.cpp")
    headers = glob.glob(os.path.join(INCLUDE, "*.h"))
    note = os.path.join(OBJDIR, os.path.basename(TORCH_LIB) + ".built_for.txt")
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:       # a torch that no package manager put there
        version = _torch_root()
    wanted = f"torch {version}, {sys.implementation.cache_tag}"
    built_for = ""
    if os.path.exists(note):
        with open(note) as f:
            built_for = f.read()
    if not force and built_for == wanted and not _stale(TORCH_LIB, [src, os.path.abspath(__file__)] + headers):
        return TORCH_LIB
    import torch
    troot = os.path.dirname(torch.__file__)
    includes = [os.path.join(troot, "include"), os.path.join(troot, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"],
                os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")]
    tmp = TORCH_LIB + f".tmp{os.getpid()}"
    # g++, which nvcc takes for its host code too, whatever $CXX says; and the C++ library that torch
    # has loaded: one linked in statically, where the compiler finds no other, is a second one in the
    # process, and its streams crash
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[a for i in includes for a in ("-isystem", i)], "-I", INCLUDE, src, "-o", tmp,
           "-L", PKG, "-lslikl", "-L", os.path.join(troot, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_cuda", "-ltorch", "-ltorch_python", "-l:libstdc++.so.6", "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"g++ failed on {src}")
    os.replace(tmp, TORCH_LIB)
    with open(note, "w") as f:
        f.write(wanted)
    return TORCH_LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
