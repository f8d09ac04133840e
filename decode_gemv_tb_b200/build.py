"""Build libtb_b200.so in-tree with nvcc for sm_100a, and _tb_bind.so beside it.

    python -m decode_gemv_tb_b200.build [--verbose]

The shared library is self-contained (static CUDA runtime) and exports only
the C interface of include/tb.h; _tb_bind.so holds the Python calls that go
through the CPython API and torch's C++ interface instead of ctypes.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libtb_b200.so")
BIND = os.path.join(PKG, "_tb_bind.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden", "-shared",
         "--expt-relaxed-constexpr", "-t", "4"]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _older(target: str, deps) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(d) > os.path.getmtime(target) for d in deps)


def _stale() -> bool:
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    deps.append(os.path.join(ROOT, "include", "tb.h"))
    return _older(LIB, deps)


def bind_tag() -> str:
    """What _tb_bind.so is built for; the file holds it, as the module's `built_for`."""
    import torch

    return f"torch {torch.__version__}, python {sys.version_info[0]}.{sys.version_info[1]}"


def _bind_stale() -> bool:
    if _older(BIND, [os.path.join(CSRC, "tb_bind.cpp"), os.path.join(ROOT, "include", "tb.h")]):
        return True
    with open(BIND, "rb") as f:
        return bind_tag().encode() + b"\0" not in f.read()


def build_bind(force: bool = False) -> str:
    """_tb_bind.so, which needs g++ and the headers of the torch that will load it."""
    if not force and not _bind_stale():
        return BIND
    if os.path.exists(BIND):  # what cannot be built anew is not left behind for another torch or another tb.h
        os.remove(BIND)
    import torch
    from torch.utils import cpp_extension

    cuda = os.path.dirname(os.path.dirname(NVCC))
    dirs = [sysconfig.get_paths()["include"], os.path.join(ROOT, "include"), os.path.join(cuda, "include"),
            *cpp_extension.include_paths()]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DTB_BUILT_FOR="{bind_tag()}"',
           *(f"-isystem{d}" for d in dirs), os.path.join(CSRC, "tb_bind.cpp"),
           "-o", BIND + ".tmp", *(f"-L{d}" for d in cpp_extension.library_paths()),
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    subprocess.run(cmd, check=True)
    os.replace(BIND + ".tmp", BIND)
    return BIND


def _build_lib(force: bool, verbose: bool):
    if not force and not _stale():
        return
    cmd = [NVCC, *ARCH, *FLAGS, "-I", os.path.join(ROOT, "include")]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    cmd += ["-o", LIB + ".tmp", *sources()]
    subprocess.run(cmd, check=True)
    os.replace(LIB + ".tmp", LIB)


def build(force: bool = False, verbose: bool = False) -> str:
    """Both libraries.  The CUDA library needs nvcc alone; without the other only the 4-bit and expert-layer calls of
    the Python binding raise, so a failure to build that one is a warning."""
    _build_lib(force, verbose)
    try:
        build_bind(force)
    except (OSError, ImportError, subprocess.CalledProcessError) as e:
        warnings.warn(f"_tb_bind.so not built, the 4-bit and expert-layer calls will raise: {e}")
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose="--verbose" in sys.argv))
