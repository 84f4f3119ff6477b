"""Build libpw.so (the C-ABI CUDA library) in-tree for sm_100a with nvcc, and _pw_binding.so (its
argument marshalling for the calls that a decoding step makes) with g++ against torch's headers."""
from __future__ import annotations

import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libpw.so")
BINDING_SRC = os.path.join(CSRC, "pw_binding.cpp")
BINDING = os.path.join(HERE, "_pw_binding.so")

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC", "-shared",
    "--expt-relaxed-constexpr",
    "-Xptxas", "-warn-spills",
]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpw.so")
    return cand


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def deps():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))) + \
        [os.path.join(ROOT, "include", "pw.h")]


def _newer(target: str, sources) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(p) <= t for p in sources)


def up_to_date() -> bool:
    return _newer(LIB, deps())


def binding_target() -> str:
    """What _pw_binding.so has to be compiled for: it uses torch's C++ classes and Python's C API."""
    return f"torch {importlib.metadata.version('torch')}, {sys.implementation.cache_tag}"


def _binding_up_to_date() -> bool:
    if not _newer(BINDING, [BINDING_SRC, os.path.join(ROOT, "include", "pw.h")]):
        return False
    with open(BINDING, "rb") as f:
        return f"[built for {binding_target()}]".encode() in f.read()


def build_binding(force: bool = False, verbose: bool = False) -> str:
    if not force and _binding_up_to_date():
        return BINDING
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    inc = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f'-DPW_BUILT_FOR="{binding_target()}"', *[f"-isystem{i}" for i in inc], BINDING_SRC, "-o", BINDING,
           "-L" + HERE, "-l:libpw.so", "-Wl,-rpath,$ORIGIN", "-L" + os.path.join(torch, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    return BINDING


def build(force: bool = False, verbose: bool = False, extra=(), binding: bool = True) -> str:
    """libpw.so, and unless binding is False (a user of the C ABI alone needs neither g++ nor torch's headers)
    the compiled part of its Python binding; what is up to date stays, unless force."""
    if force or not up_to_date():
        cmd = [nvcc(), *NVCC_FLAGS, *extra, "-I", os.path.join(ROOT, "include"), "-o", LIB, *sources()]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        subprocess.run(cmd, check=True)
    if binding:
        build_binding(force=force, verbose=verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, binding="--no-binding" not in sys.argv,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
    print(LIB)
