"""Build the CUDA library (liblosa.so) for sm_100a with nvcc, and the Python side's argument marshalling (_binding.so) with
the host compiler, in-tree."""
from __future__ import annotations

import glob
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "liblosa.so")
BINDING = os.path.join(PKG, "_binding.so")


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  [os.path.join(INCLUDE, "losa.h")])


def command(out: str = LIB, extra=()):
    return [nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
            "-Xcompiler", "-fPIC", "-shared", "-I" + INCLUDE, *extra, "-o", out, os.path.join(CSRC, "losa.cu")]


def build(force: bool = False, verbose: bool = False) -> str:
    stale = not os.path.exists(LIB) or any(os.path.getmtime(s) > os.path.getmtime(LIB) for s in sources())
    if force or stale:
        tmp = LIB + ".tmp"
        cmd = command(tmp, ("-Xptxas", "-v") if verbose else ())
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB)
    build_binding()
    return LIB


def binding_command(out: str = BINDING):
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    includes = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                os.path.join(cuda, "include"), sysconfig.get_paths()["include"], INCLUDE]
    libs = [os.path.join(root, "lib")]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-I{i}" for i in includes],
            os.path.join(CSRC, "binding.cpp"), "-o", out, *[f"-L{p}" for p in libs], "-ltorch_python", "-ltorch", "-ltorch_cpu",
            "-lc10", "-lc10_cuda"]


def build_binding(force: bool = False) -> str:
    needs = [os.path.join(CSRC, "binding.cpp"), os.path.join(INCLUDE, "losa.h")]
    if force or not os.path.exists(BINDING) or any(os.path.getmtime(s) > os.path.getmtime(BINDING) for s in needs):
        tmp = BINDING + ".tmp"
        subprocess.run(binding_command(tmp), check=True)
        os.replace(tmp, BINDING)
    return BINDING


if __name__ == "__main__":
    print(build(force=True, verbose=True))
    print(build_binding(force=True))
