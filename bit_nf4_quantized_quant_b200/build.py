"""Builds libqlora_nf4.so (nvcc, sm_100a) and the Python binding _step.so over it (g++), in-tree.

    python -m bit_nf4_quantized_quant_b200.build [--force] [--verbose]
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC_DIR = os.path.join(HERE, "csrc")
MAIN = os.path.join(SRC_DIR, "qlora_nf4.cu")
LIB = os.path.join(HERE, "libqlora_nf4.so")
BINDING_SRC = os.path.join(SRC_DIR, "binding.cpp")
BINDING = os.path.join(HERE, "_step.so")
HEADER = os.path.join(ROOT, "include", "qlora_nf4.h")

NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
              "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC", "-shared", "-Xcompiler", "-fvisibility=hidden"]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.sep not in c or os.path.exists(c)):
            return c
    return "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(SRC_DIR, "*.cu")) + glob.glob(os.path.join(SRC_DIR, "*.cuh"))) + [HEADER]


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in sources())


def _torch_stamp() -> str:
    """What the binding carries of the torch it was built with, whose C++ interface differs from version to version."""
    import torch
    return f"built with torch {torch.__version__};"


def _binding_stale() -> bool:
    if not os.path.exists(BINDING):
        return True
    t = os.path.getmtime(BINDING)
    if any(os.path.getmtime(s) > t for s in (BINDING_SRC, HEADER)):
        return True
    with open(BINDING, "rb") as f:
        return _torch_stamp().encode() not in f.read()


def build_binding(force: bool = False) -> str:
    """The CPython extension over libqlora_nf4.so (which it finds beside itself)."""
    if not force and not _binding_stale():
        return BINDING
    import sysconfig

    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    tlib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.dirname(os.path.dirname(_nvcc())) if os.path.sep in _nvcc() else "/usr/local/cuda"
    tmp = f"{BINDING}.tmp{os.getpid()}"
    subprocess.check_call(
        ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
         f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", f'-DQLORA_TORCH_STAMP="{_torch_stamp()}"',
         f"-I{sysconfig.get_paths()['include']}",
         f"-I{inc}", f"-I{os.path.join(inc, 'torch', 'csrc', 'api', 'include')}", f"-I{os.path.join(cuda, 'include')}",
         BINDING_SRC, "-o", tmp, f"-L{HERE}", "-l:libqlora_nf4.so", "-Wl,-rpath,$ORIGIN", f"-L{tlib}", "-lc10",
         "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"])
    os.replace(tmp, BINDING)
    return BINDING


def build(force: bool = False, verbose: bool = False, extra=None) -> str:
    _build_lib(force, verbose, extra)
    build_binding(force)
    return LIB


def _build_lib(force: bool, verbose: bool, extra) -> str:
    if not force and not stale():
        return LIB
    tmp = f"{LIB}.tmp{os.getpid()}"            # per process: concurrent builds never share a file
    cmd = [_nvcc(), *NVCC_FLAGS, *(extra or []), MAIN, "-o", tmp]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB)
