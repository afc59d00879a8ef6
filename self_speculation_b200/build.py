"""Build the CUDA library `libnld.so` in-tree with nvcc for sm_100a, and `_operators.so`, the Python
entry of its operators on torch tensors, with g++.

Usage: python -m self_speculation_b200.build   (or build() from Python)
Sources: self_speculation_b200/csrc/*.cu, public header include/nld.h.
"""
from __future__ import annotations

import importlib.metadata
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libnld.so")
OPERATORS = os.path.join(PKG, "_operators.so")
SOURCES = ["nld_api.cu", "gemm_tc.cu", "gemm_simt.cu", "attention.cu", "decode_kernels.cu",
           "attention_small.cu", "attention_wide.cu", "qkv_write.cu", "sampling.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _run(cmd, what: str, verbose: bool) -> subprocess.CompletedProcess:
    if verbose:
        print(" ".join(cmd))
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n" + r.stdout + r.stderr)
    return r


def operators_built_for() -> str:
    """The Python and torch whose binary interfaces `_operators.so` is built against; the file holds this text."""
    return f"built for {sysconfig.get_config_var('SOABI')}, torch {importlib.metadata.version('torch')};"


def _operators_stale(target: str, deps) -> bool:
    if _stale(target, deps):
        return True
    with open(target, "rb") as f:
        return operators_built_for().encode() not in f.read()


def _build_operators(force: bool, verbose: bool) -> None:
    source = os.path.join(CSRC, "bind_operators.cpp")
    if not force and not _operators_stale(OPERATORS, [source, os.path.join(ROOT, "include", "nld.h")]):
        return
    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    paths = [os.path.join(ROOT, "include"), *include_paths(), os.path.join(cuda, "include"), sysconfig.get_path("include")]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DNLD_BUILT_FOR="{operators_built_for()}"', source, "-o", OPERATORS + ".tmp"]
    for p in paths:
        cmd += ["-isystem" if p != paths[0] else "-I", p]
    cmd += [f"-L{p}" for p in library_paths()]
    cmd += [f"-L{PKG}", "-l:libnld.so", "-Wl,-rpath,$ORIGIN", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    _run(cmd, "g++", verbose)
    os.replace(OPERATORS + ".tmp", OPERATORS)


def build(force: bool = False, verbose: bool = False, ptxas_v: bool = False) -> str:
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if not f.endswith(".cpp")]
    if force or _stale(LIB, deps + [os.path.join(ROOT, "include", "nld.h")]):
        _build_library(verbose, ptxas_v)
    _build_operators(force, verbose)
    return LIB


def _build_library(verbose: bool, ptxas_v: bool) -> None:
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "--shared", "-Xcompiler", "-fPIC", "--threads", "0",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-o", LIB + ".tmp"]
    if ptxas_v:
        cmd += ["-Xptxas", "-v"]
    cmd += [os.path.join(CSRC, s) for s in SOURCES]
    cmd += ["-lcudart"]
    r = _run(cmd, "nvcc", verbose)
    if verbose or ptxas_v:
        sys.stdout.write(r.stdout + r.stderr)
    os.replace(LIB + ".tmp", LIB)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_v="-v" in sys.argv)
