"""Build libmoe_ffn.so in-tree for sm_100a with nvcc, and the Python module behind ops.py.

Usage: ``python -m mixture_experts_ffn_expert_b200.build`` (or ``build()``).
The libraries land in ``mixture_experts_ffn_expert_b200/lib/`` next to the
binding that loads them. nvcc cross-compiles, so no GPU is needed to build.
"""
from __future__ import annotations

import importlib.metadata
import importlib.util
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

HOST_NAME = "_moe_host.so"
HOST_SOURCE = "host_ops.cpp"
STAMP_SUFFIX = ".built-with"      # beside the module: the torch and Python it was compiled against

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


def host_path() -> str:
    return os.path.join(LIBDIR, HOST_NAME)


def _stale(target: str, sources) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    deps = [os.path.join(CSRC, s) for s in sources]
    deps.append(os.path.join(INCLUDE, "moe_ffn.h"))
    deps.append(os.path.abspath(__file__))
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Compile the CUDA library and the module behind ops.py (each skipped when it is newer
    than its sources). Returns the CUDA library's path. The C ABI needs the library alone: where
    torch or a C++ compiler is absent, the module is left out with a message (and ops.py, which
    needs it, raises when it is called)."""
    target = _build_library(force, verbose, extra_flags)
    _build_host(force, verbose)
    return target


def _torch_tag() -> str:
    """The torch and Python that a module is compiled against ("" without torch)."""
    if importlib.util.find_spec("torch") is None:
        return ""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        import torch
        version = torch.__version__
    return f"torch {version}, {sys.implementation.cache_tag}"


def _host_stale(target: str, tag: str) -> bool:
    if _stale(target, [HOST_SOURCE]):
        return True
    try:
        with open(target + STAMP_SUFFIX) as f:
            return f.read() != tag
    except OSError:
        return True


def _build_host(force: bool, verbose: bool) -> None:
    """The torch-facing module: plain C++ against torch's headers, linked to the library."""
    target = host_path()
    tag = _torch_tag()
    compiler = os.environ.get("CXX", "g++")
    missing = "torch" if not tag else compiler if shutil.which(compiler) is None else None
    if missing:
        print(f"{HOST_NAME} is not built: {missing} was not found (the torch functions of "
              "ops.py need it, the C ABI does not)", file=sys.stderr)
        return
    if not force and not _host_stale(target, tag):
        return
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    tmp = target + ".tmp"
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda_include = os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include")
    includes = [INCLUDE, *cpp_extension.include_paths(), sysconfig.get_paths()["include"],
                cuda_include]
    cmd = [compiler, "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f"-I{i}" for i in includes], os.path.join(CSRC, HOST_SOURCE), "-o", tmp,
           f"-L{LIBDIR}", f"-l:{LIBNAME}", "-Wl,-rpath,$ORIGIN", f"-L{torch_lib}",
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, target)
    with open(target + STAMP_SUFFIX, "w") as f:
        f.write(tag)


def _build_library(force: bool, verbose: bool, extra_flags) -> str:
    target = lib_path()
    if not force and not _stale(target, SOURCES + HEADERS):
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
