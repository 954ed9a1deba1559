"""Build the CUDA library kv_cache_retrieval_b200/libhhr.so for sm_100a.

Usage: ``python -m kv_cache_retrieval_b200.build [--force] [--verbose]``.
Sources are compiled in parallel with nvcc, then linked into one shared
library with a static CUDA runtime.
"""
from __future__ import annotations

import os
import re
import subprocess
import sys
import time
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libhhr.so")
SOURCES = ["api.cu", "decode.cu", "encode.cu", "noalloc.cu", "paged.cu", "paged_bf16.cu", "paged_bf16_e4m3.cu",
           "paged_f16.cu", "paged_f16_e4m3.cu", "rope.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
           "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _deps() -> list[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "hhr.h"))
    files.append(os.path.abspath(__file__))
    return files


def _src_deps(src: str) -> list[str]:
    """A source file and the files of this tree it includes, directly or not."""
    seen, todo = [], [os.path.join(CSRC, src)]
    while todo:
        f = todo.pop()
        if f in seen:
            continue
        seen.append(f)
        with open(f) as fh:
            names = re.findall(r'^#include "([^"]+)"', fh.read(), flags=re.M)
        todo += [p for n in names for p in (os.path.join(CSRC, n), os.path.join(INCLUDE, n)) if os.path.exists(p)]
    return seen + [os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _deps())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    begun = time.time()
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if verbose else []

    def put(made: str, to: str, t: float) -> None:
        """A whole file, as old as the sources it was made of may be: one saved in the meantime is newer."""
        os.utime(made, (t, t))
        os.replace(made, to)

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        if not force and os.path.exists(obj) and all(os.path.getmtime(f) < os.path.getmtime(obj)
                                                     for f in _src_deps(src)):
            return obj
        t, made = time.time(), obj + ".tmp.o"
        cmd = [nvcc, *ARCH, *NVFLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", made]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stderr)
        put(made, obj, t)
        return obj

    with ThreadPoolExecutor(len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    put(tmp, LIB, begun)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
