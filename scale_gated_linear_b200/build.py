"""Build the MS-GLA CUDA library (libmsgla.so) in-tree for sm_100a.

Usage: python -m scale_gated_linear_b200.build [--force] [--verbose]
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libmsgla.so")
SOURCES = ["msgla_abi.cu", "k_gemm.cu", "k_gla.cu", "k_aux.cu", "k_pool.cu", "k_decode.cu", "k_scan.cu", "k_norm.cu",
           "ops_abi.cu"]
HEADERS = ["msgla_internal.h", "ops_internal.h", "sm100_ptx.cuh"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(ROOT, "include", "msgla.h")]
    return any(os.path.getmtime(p) > t for p in deps)


def _run(cmd: list, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or res.returncode != 0:
        sys.stdout.write(res.stdout)
        sys.stderr.write(res.stderr)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed with exit code {res.returncode}")


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    flags = [*ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include")]
    with tempfile.TemporaryDirectory() as tmp, ThreadPoolExecutor(os.cpu_count() or 1) as pool:
        objects = [os.path.join(tmp, f + ".o") for f in SOURCES]
        # one nvcc a source, at once: one for all of them takes the sources one after another
        jobs = [pool.submit(_run, [nvcc(), *(["-Xptxas=-v"] if verbose else []), *flags, "-c", os.path.join(CSRC, f), "-o", o],
                            verbose) for f, o in zip(SOURCES, objects)]
        for job in jobs:
            job.result()
        _run([nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", LIB + ".tmp", *objects], verbose)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB)
