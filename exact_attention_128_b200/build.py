"""Build the in-tree CUDA library ``libfa_b200.so`` for sm_100a with nvcc, and ``_binding.so``.

The library is a single translation unit (``csrc/fa_api.cu`` includes the kernels) and
links the CUDA runtime statically, so it loads on hosts without a GPU; the driver's
TMA descriptor encoder is looked up at run time.  ``_binding.so`` is the host code that
checks tensors and allocates outputs for some of the Python calls (``csrc/binding.cpp``,
compiled against the installed torch); it links neither the library nor a kernel.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libfa_b200.so")
BINDING = os.path.join(HERE, "_binding.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfa_b200.so")


def sources():
    out = []
    for root in (CSRC, os.path.join(os.path.dirname(HERE), "include")):
        for f in sorted(os.listdir(root)):
            if f.endswith((".cu", ".cuh", ".h")):
                out.append(os.path.join(root, f))
    return out


def up_to_date(target: str = LIB, files=None) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(s) <= t for s in (sources() if files is None else files))


def build_binding(force: bool = False) -> str:
    import sysconfig

    import torch

    source = os.path.join(CSRC, "binding.cpp")
    files = [source, os.path.join(os.path.dirname(HERE), "include", "fa.h"), torch.__file__]
    if not force and up_to_date(BINDING, files):
        return BINDING
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    cmd = [
        shutil.which("g++") or "c++",
        "-O2",
        "-std=c++17",
        "-fPIC",
        "-shared",
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
        *("-I" + i for i in include),
        source,
        "-L" + os.path.join(root, "lib"),
        *("-l" + name for name in ("torch_python", "torch_cpu", "c10_cuda", "c10")),
        "-o",
        BINDING + ".tmp",
    ]
    subprocess.run(cmd, check=True)
    os.replace(BINDING + ".tmp", BINDING)
    return BINDING


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """The library, which needs nvcc alone, and then the binding (left out on a host without torch)."""
    if force or not up_to_date():
        build_library(verbose, extra_flags)
    if importlib.util.find_spec("torch"):
        build_binding(force)
    else:
        print("torch is not installed: _binding.so, the Python side of some calls, is not built", file=sys.stderr)
    return LIB


def build_library(verbose: bool = False, extra_flags=()) -> str:
    cmd = [
        nvcc_path(),
        *ARCH,
        "-O3",
        "-std=c++17",
        "-lineinfo",
        "-Xcompiler",
        "-fPIC",
        "-shared",
        *extra_flags,
        "-o",
        LIB + ".tmp",
        os.path.join(CSRC, "fa_api.cu"),
    ]
    if verbose:
        cmd.insert(-3, "-Xptxas=-v")
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
