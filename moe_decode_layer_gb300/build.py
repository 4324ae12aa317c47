"""Build the C-ABI shared library (libmoe_decode.so) for sm_103a with nvcc.

Each translation unit compiles in its own nvcc process (in parallel); the objects
are linked with nvcc into ``moe_decode_layer_gb300/lib/libmoe_decode.so``.
Rebuilds only when a source is newer than the library. No CMake, no torch
extension machinery: the library has a plain C ABI.

    python -m moe_decode_layer_gb300.build [--force] [--verbose]
"""

from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libmoe_decode.so")

DECODE_SOURCES = ["api.cu", "kernels_bf16.cu", "kernels_nvfp4.cu", "kernels_fp8.cu", "kernels_flat.cu", "kernels_sk.cu",
                  "static_run.cu"]
ROWS_SOURCES = ["rows_api.cu", "rows_kernels.cu", "rows_route.cu", "rows_gemm.cu", "rows_gemm_fp8.cu",
                "rows_gemm_nvfp4.cu", "dense_api.cu", "dense_quantise.cu",
                "dense_stream.cu", "dense_gemm.cu",
                "dense_gemm_backward.cu", "dense_gemm_int8.cu", "dense_lanes.cu"]
SOURCES = DECODE_SOURCES + ROWS_SOURCES
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
         "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the MoE decode library")


def _deps() -> list[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files.append(os.path.abspath(__file__))
    return files


def sources_of(units: list[str]) -> list[str]:
    """Names of these translation units and of every header of csrc/ that they include, sorted."""
    todo, found = list(units), set()
    while todo:
        name = todo.pop()
        if name in found or not os.path.exists(os.path.join(CSRC, name)):
            continue
        found.add(name)
        with open(os.path.join(CSRC, name)) as f:
            todo += re.findall(r'^\s*#include "([^"]+)"', f.read(), re.M)
    return sorted(n for n in found if os.sep not in n)


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _deps())


def _compile(src: str, verbose: bool, ptxas_verbose: bool) -> str:
    obj = os.path.join(BUILD, src.replace(".cu", ".o"))
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if ptxas_verbose:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode != 0 or ptxas_verbose:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}")
    return obj


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile and link the library if needed; return its path."""
    if not force and not ptxas_verbose and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose, ptxas_verbose), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "--cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        raise RuntimeError("linking libmoe_decode.so failed")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-verbose", action="store_true")
    a = ap.parse_args()
    print(build(a.force, a.verbose, a.ptxas_verbose))
