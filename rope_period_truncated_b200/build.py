"""Build libwaveprune.so in-tree with nvcc for sm_100a, and _calls.so, the
compiled Python binding of the serving calls, with the C++ compiler against
torch's headers.

Usage: ``python -m rope_period_truncated_b200.build`` (or ``build()``).
The library links the CUDA runtime statically and reaches the driver's
tensor-map encoder through the runtime's entry-point query, so it loads on a
machine without a GPU driver (calls then return WP_ERR_CUDA).
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libwaveprune.so")
BINDING = os.path.join(PKG, "_calls.so")
BINDING_SOURCE = os.path.join(CSRC, "wp_torch.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-rdc=true",
    "-Xcompiler", "-fPIC,-fvisibility=default",
    "--expt-relaxed-constexpr",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(p) > t for p in deps)


def _binding_stale(made_for: str) -> bool:
    """Is the binding absent, older than its sources, or built against another torch or Python, whose ABI it would not fit?"""
    if not os.path.exists(BINDING) or not os.path.exists(_binding_note()):
        return True
    with open(_binding_note()) as f:
        if f.read() != made_for:
            return True
    deps = (BINDING_SOURCE, os.path.join(INCLUDE, "waveprune.h"))
    return any(os.path.getmtime(p) > os.path.getmtime(BINDING) for p in deps)


def _binding_note() -> str:
    return os.path.join(os.path.dirname(BINDING), "_build", "calls.txt")


def _build_binding(force: bool, verbose: bool) -> None:
    import torch
    made_for = f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}\n"
    if not force and not _binding_stale(made_for):
        return
    from torch.utils import cpp_extension
    include = [f for p in cpp_extension.include_paths("cuda") for f in ("-isystem", p)]
    libs = [f for p in cpp_extension.library_paths("cuda") for f in ("-L", p)]
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I", INCLUDE,
           "-isystem", sysconfig.get_paths()["include"], *include, BINDING_SOURCE, "-o", tmp, *libs,
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, BINDING)
    os.makedirs(os.path.dirname(_binding_note()), exist_ok=True)
    with open(_binding_note(), "w") as f:
        f.write(made_for)


def _build_library(force: bool, verbose: bool, extra_flags) -> None:
    if not force and not _stale():
        return
    nvcc = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *NVCC_FLAGS, *extra_flags, "-I", INCLUDE, "-I", CSRC, "-shared", *sources(), "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """The library first: it needs no torch headers, and all calls but the serving ones need no binding."""
    _build_library(force, verbose, extra_flags)
    _build_binding(force, verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
