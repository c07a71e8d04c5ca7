"""Build libmoe_ffn.so in-tree for sm_100a with nvcc.

Usage: ``python -m mixture_experts_ffn_expert_b200.build`` (or ``build()``).
The library lands in ``mixture_experts_ffn_expert_b200/lib/`` next to the
binding that loads it. nvcc cross-compiles, so no GPU is needed to build.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIBDIR = os.path.join(PKG, "lib")
LIBNAME = "libmoe_ffn.so"
SOURCES = ["moe_ffn.cu", "gated_ffn.cu", "ops.cu"]
HEADERS = ["ptx_sm100.cuh", "gemm_sm100.cuh", "route.cuh", "router_sm100.cuh",
           "dense_gemm_sm100.cuh", "stream_gemm_sm100.cuh", "norm.cuh", "dropout.cuh", "ops_types.cuh", "ops_host.h"]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "--expt-relaxed-constexpr", "--threads", "0",
]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: set NVCC or put the CUDA toolkit on PATH")


def lib_path() -> str:
    return os.path.join(LIBDIR, LIBNAME)


def _stale(target: str) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    deps = [os.path.join(CSRC, s) for s in SOURCES + HEADERS]
    deps.append(os.path.join(INCLUDE, "moe_ffn.h"))
    deps.append(os.path.abspath(__file__))
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Compile the CUDA library (skipped when it is newer than its sources)."""
    target = lib_path()
    if not force and not _stale(target):
        return target
    os.makedirs(LIBDIR, exist_ok=True)
    tmp = target + ".tmp"
    cmd = [nvcc_path(), *NVCC_FLAGS, *(extra_flags or []), f"-I{INCLUDE}", f"-I{CSRC}",
           *[os.path.join(CSRC, s) for s in SOURCES], "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
    if verbose and (res.stdout or res.stderr):
        print(res.stdout, res.stderr, sep="\n", file=sys.stderr)
    os.replace(tmp, target)
    return target


if __name__ == "__main__":
    force = "--force" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None
    print(build(force=force or bool(extra), verbose=True, extra_flags=extra))
