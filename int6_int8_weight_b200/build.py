"""Build libgq.so (the CUDA kernels and the C ABI of include/gq.h) in-tree.

    python -m int6_int8_weight_b200.build

Compiles for sm_100a only, with -fmad=false so that no floating-point
multiply and add is contracted into a fused operation (the rounding-critical
steps also use explicit-rounding intrinsics).
"""
from __future__ import annotations

import os
import re
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libgq.so")
OBJ = os.path.join(PKG, "_build")
SOURCES = [os.path.join(CSRC, f) for f in ("gq_api.cu", "gq_linear.cu", "gq_adamw.cu")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] + \
    [os.path.join(INCLUDE, "gq.h")]

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-fmad=false",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _deps(path: str, seen: set) -> set:
    """`path` and the library's own headers that it includes, directly or not."""
    if path not in seen:
        seen.add(path)
        with open(path) as f:
            for name in re.findall(r'^#include "([\w./]+)"', f.read(), re.M):
                for d in (CSRC, INCLUDE):
                    if os.path.exists(os.path.join(d, name)):
                        _deps(os.path.join(d, name), seen)
    return seen


def build(force: bool = False, verbose: bool = False) -> str:
    if (not force and os.path.exists(LIB)
            and os.path.getmtime(LIB) >= max(os.path.getmtime(d) for d in DEPS)):
        return LIB
    # one object per source whose own files changed, compiled side by side, then one link
    os.makedirs(OBJ, exist_ok=True)
    objs, jobs = [], []
    for src in SOURCES:
        obj = os.path.join(OBJ, os.path.basename(src) + ".o")
        objs.append(obj)
        if (not force and os.path.exists(obj)
                and os.path.getmtime(obj) >= max(os.path.getmtime(d) for d in _deps(src, set()) | {__file__})):
            continue
        tmp = obj + f".tmp{os.getpid()}"
        cmd = [nvcc(), *(["-Xptxas=-v"] if verbose else []), *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src,
               "-o", tmp]
        if verbose:
            print(" ".join(cmd))
        jobs.append((cmd, tmp, obj, subprocess.Popen(cmd)))
    status = [job.wait() for _, _, _, job in jobs]
    for (cmd, tmp, obj, _), rc in zip(jobs, status):
        if rc != 0:
            raise subprocess.CalledProcessError(rc, cmd)
        os.replace(tmp, obj)
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run([nvcc(), "--shared", *NVCC_FLAGS, *objs, "-o", tmp], check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
