"""Builds the CUDA library ``libfgm.so`` in the package directory with nvcc
for sm_103a (one process per translation unit, side by side; no cmake)."""

from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libfgm.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h")))


def units() -> list[str]:
    return [f for f in sources() if f.endswith(".cu")]


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    """Compile csrc/*.cu into libfgm.so unless it is newer than every source."""
    srcs = sources() + [os.path.join(ROOT, "include", "fgm.h")]
    if not force and os.path.exists(LIB) and all(os.path.getmtime(LIB) >= os.path.getmtime(s) for s in srcs):
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    flags = [*(extra or []), *(["-Xptxas=-v"] if verbose else []), *ARCH, "-O3", "-lineinfo", "-std=c++17",
             "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include")]
    objs = [f"{tmp}.{i}.o" for i in range(len(units()))]
    try:
        procs = [subprocess.Popen([nvcc(), *flags, "-c", "-o", o, u]) for u, o in zip(units(), objs)]
        codes = [p.wait() for p in procs]
        if any(codes):
            raise subprocess.CalledProcessError(next(c for c in codes if c), nvcc())
        subprocess.run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs], check=True)
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
