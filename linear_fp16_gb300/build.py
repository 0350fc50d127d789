"""Build the CUDA library libpoot_linear.so (sm_103a) in-tree with nvcc, and
the extension that calls it on torch tensors.

Usage: python -m linear_fp16_gb300.build [--verbose]
builds the library, and the extension where torch is installed.  Both land in
linear_fp16_gb300/_build/ (git-ignored).  The library needs neither torch nor
Python's headers, to be built or to be loaded.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
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

EXT_SOURCE = os.path.join(CSRC, "ffn_torch.cpp")
EXT_DEPENDS = [EXT_SOURCE] + [os.path.join(INCLUDE, f) for f in ("poot_linear.h", "poot_ffn.h")]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
         "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpoot_linear.so")
    return cand


def extension() -> str:
    """Path of the tensor-level extension, built for this torch and interpreter."""
    import torch
    return os.path.join(BUILD, f"_ffn_torch.{sys.implementation.cache_tag}.{torch.__version__}.so")


def _newer(target: str, deps) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(p) <= t for p in deps)


def up_to_date() -> bool:
    """Whether the library is built from the present sources (torch plays no part in it)."""
    return _newer(LIB, DEPENDS)


def extension_up_to_date() -> bool:
    return _newer(extension(), EXT_DEPENDS)


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
    """The C library: nvcc alone, no torch and no Python headers."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    tag = f".tmp{os.getpid()}"
    objs = [os.path.join(BUILD, os.path.basename(src) + tag + ".o") for src in SOURCES]
    lib = LIB + tag
    compiles = [[nvcc(), *ARCH, *FLAGS, "-Xptxas=-v", "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", o]
                for src, o in zip(SOURCES, objs)]
    try:
        # the translation units side by side, then the link
        with ThreadPoolExecutor(len(compiles)) as pool:
            list(pool.map(lambda cmd: _run(cmd, verbose), compiles))
        _run([nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", *objs, "-o", lib], verbose)
        os.replace(lib, LIB)
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)
    return LIB


def build_extension(force: bool = False, verbose: bool = False) -> str:
    """The extension for torch tensors, and the library it links to (side by side)."""
    ext = extension()
    if not force and up_to_date() and extension_up_to_date():
        return ext
    import torch
    os.makedirs(BUILD, exist_ok=True)
    tag = f".tmp{os.getpid()}"
    obj, out = os.path.join(BUILD, os.path.basename(EXT_SOURCE) + tag + ".o"), ext + tag
    tdir = os.path.dirname(torch.__file__)
    includes = [INCLUDE, os.path.join(tdir, "include"), os.path.join(tdir, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"],
                os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")]
    try:
        with ThreadPoolExecutor(2) as pool:
            jobs = [pool.submit(build, force, verbose),
                    pool.submit(_run, ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
                                       *[f"-I{p}" for p in includes], "-c", EXT_SOURCE, "-o", obj], verbose)]
            for job in jobs:
                job.result()
        # (the loader finds the library beside the extension; torch is loaded already)
        _run(["g++", "-shared", obj, "-L" + BUILD, "-l:" + os.path.basename(LIB), "-L" + os.path.join(tdir, "lib"),
              "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", "-o", out], verbose)
        os.replace(out, ext)
    finally:
        if os.path.exists(obj):
            os.remove(obj)
    return ext


if __name__ == "__main__":
    print(build(force=True, verbose="--verbose" in sys.argv))
    if importlib.util.find_spec("torch") is not None:
        print(build_extension(force=not extension_up_to_date(), verbose="--verbose" in sys.argv))
