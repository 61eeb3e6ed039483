"""Build the C-ABI library libttt.so in-tree with nvcc for sm_100a.

    python -m test_weight_layers_b200.build [--force] [--verbose]

The library is a few translation units (UNITS below) compiled side by side and
linked with the CUDA runtime statically, so it needs nothing at run time
beyond the NVIDIA driver.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libttt.so")
UNITS = ["ttt_capi.cu", "ttt_delta.cu", "ttt_norm.cu"]
OBJ = os.path.join(PKG, "_build")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found; set NVCC or put the CUDA toolkit on PATH")


def _sources():
    out = [os.path.join(INCLUDE, "ttt.h")]
    for f in sorted(os.listdir(CSRC)):
        if f.endswith((".cu", ".cuh", ".h")):
            out.append(os.path.join(CSRC, f))
    return out


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(s) <= t for s in _sources())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJ, exist_ok=True)

    def run(args, what):
        res = subprocess.run([nvcc(), *ARCH, *args], capture_output=True, text=True)
        if verbose or res.returncode != 0:
            sys.stderr.write(res.stdout + res.stderr)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed {what}")

    def compile_unit(unit):
        src, obj = os.path.join(CSRC, unit), os.path.join(OBJ, unit + ".o")
        # an object newer than its unit and every header is kept
        deps = [src] + [f for f in _sources() if not f.endswith(".cu")]
        if force or not os.path.exists(obj) or any(os.path.getmtime(d) > os.path.getmtime(obj) for d in deps):
            flags = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC,-O2",
                     "-I", INCLUDE, "-I", CSRC] + (["-Xptxas", "-v"] if verbose else [])
            run([*flags, "-c", "-o", obj + ".tmp", src], f"compiling {unit}")
            os.replace(obj + ".tmp", obj)
        return obj

    with concurrent.futures.ThreadPoolExecutor(len(UNITS)) as pool:
        objects = list(pool.map(compile_unit, UNITS))
    run(["-shared", "-cudart", "static", "-Xcompiler", "-fPIC", "-o", LIB + ".tmp", *objects], "linking libttt.so")
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB)
