"""Build libnvfp4.so in-tree with nvcc for sm_100a (no JIT cache)."""
from __future__ import annotations

import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libnvfp4.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "--expt-relaxed-constexpr",
    "-Xptxas", "-warn-spills",
    "-I", INCLUDE, "-I", CSRC,
]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def attention_sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "attention", "*.cu")))


BINDING_SOURCE = os.path.join(CSRC, "binding", "attention_binding.cpp")


def binding_path(torch_version: str, python_tag: str = sys.implementation.cache_tag) -> str:
    """Where the marshalling module for one torch and one Python lies: it is
    linked to both, so one that was built for others is not found."""
    return os.path.join(PKG, f"_attention-{python_tag}-torch{torch_version}.so")


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """The CPython module that marshals the attention layer's arguments (torch
    headers; linked to torch and Python only)."""
    import sysconfig
    import torch
    from torch.utils import cpp_extension
    path = binding_path(torch.__version__)
    inputs = [BINDING_SOURCE, os.path.join(INCLUDE, "nvfp4.h")]
    if not force and os.path.exists(path) and all(os.path.getmtime(d) <= os.path.getmtime(path) for d in inputs):
        return path
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = path + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-I", os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"),
           *[a for d in cpp_extension.include_paths() for a in ("-isystem", d)], BINDING_SOURCE, "-o", tmp,
           "-L", libs, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(tmp, path)
    return path


def deps() -> list[str]:
    headers = [f for d in (CSRC, os.path.join(CSRC, "attention")) for ext in ("*.cuh", "*.h")
               for f in sorted(glob.glob(os.path.join(d, ext)))]
    return sources() + attention_sources() + headers + [os.path.join(INCLUDE, "nvfp4.h")]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in deps())


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None, binding: bool = True) -> str:
    """The library and, unless `binding` is false, the attention layer's
    marshalling module, which ops.py needs and a caller of the C ABI does not
    (nor torch's headers and g++).  The library comes first."""
    build_library(force, verbose, extra)
    if binding:
        build_binding(force, verbose)
    return LIB


def build_library(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    if not force and up_to_date():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, *NVCC_FLAGS, *(extra or []), "-o", tmp, *sources(), *attention_sources()]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None, binding="--library-only" not in sys.argv)
    print(LIB)
