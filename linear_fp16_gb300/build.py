"""Build the CUDA library libpoot_linear.so (sm_103a) in-tree with nvcc.

Usage: python -m linear_fp16_gb300.build [--verbose]
The library lands in linear_fp16_gb300/_build/ (git-ignored).
"""
from __future__ import annotations

import os
import re
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libpoot_linear.so")
SOURCES = [os.path.join(CSRC, f) for f in ("poot_linear.cu", "poot_ffn.cu")]
DEPENDS = SOURCES + [os.path.join(CSRC, f) for f in (
    "ptx.cuh", "gemm_tcgen05.cuh", "gemv.cuh", "epilogue.cuh", "splitk.cuh", "pack.cuh", "shards.cuh", "host.cuh",
    "mma.cuh", "ffn_gemm.cuh", "ffn_gemv.cuh", "ffn_elem.cuh", "clip.cuh")] + [
    os.path.join(INCLUDE, f) for f in ("poot_linear.h", "poot_ffn.h")]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
         "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpoot_linear.so")
    return cand


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in DEPENDS)


def _run(cmd, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stdout.write(r.stdout)
        sys.stderr.write(r.stderr)
    if r.returncode != 0:
        raise subprocess.CalledProcessError(r.returncode, cmd)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    tag = f".tmp{os.getpid()}"
    objs = [os.path.join(BUILD, os.path.basename(src) + tag + ".o") for src in SOURCES]
    tmp = LIB + tag
    compiles = [[nvcc(), *ARCH, *FLAGS, "-Xptxas=-v", "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", o]
                for src, o in zip(SOURCES, objs)]
    link = [nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", *objs, "-o", tmp]
    try:
        # the translation units side by side, then the link
        with ThreadPoolExecutor(len(compiles)) as pool:
            list(pool.map(lambda cmd: _run(cmd, verbose), compiles))
        _run(link, verbose)
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose="--verbose" in sys.argv))
