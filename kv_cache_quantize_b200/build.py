"""Build libkvq.so, the sm_100a CUDA library behind include/kvq.h.

nvcc cross-compiles for sm_100a without a GPU.  -fmad=false keeps every
binary32 multiply and add separately rounded (the kernels also use the
explicitly rounded intrinsics); the CUDA runtime is linked statically so the
library only needs the driver.
"""
import os
import re
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libkvq.so")
OBJ = os.path.join(HERE, "_build")
SOURCES = [os.path.join(CSRC, f) for f in ("kvq.cu", "attention.cu", "pages.cu")]
NVCC = os.environ.get("NVCC", "nvcc")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17", "-fmad=false",
         "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "-cudart", "static",
         "-I", os.path.join(ROOT, "include")]


def _deps(path, seen=None):
    """A source file and every file of this repository that it includes."""
    seen = set() if seen is None else seen
    if path not in seen:
        seen.add(path)
        with open(path, encoding="utf-8") as f:
            names = re.findall(r'^#include "([^"]+)"', f.read(), flags=re.M)
        for n in names:
            for d in (CSRC, os.path.join(ROOT, "include")):
                if os.path.exists(os.path.join(d, n)):
                    _deps(os.path.join(d, n), seen)
    return seen


def _stale(target, deps) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(p) > os.path.getmtime(target) for p in deps)


def needs_build() -> bool:
    return _stale(LIB, {os.path.abspath(__file__)}.union(*(_deps(s) for s in SOURCES)))


def build(force: bool = False, verbose: bool = False) -> str:
    if not (force or needs_build()):
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    tag = f".tmp{os.getpid()}"
    objects, jobs = [], []
    for s in SOURCES:                    # the units compile side by side, then link into one library
        o = os.path.join(OBJ, os.path.basename(s)[:-3] + ".o")
        objects.append(o)
        if force or _stale(o, _deps(s) | {os.path.abspath(__file__)}):
            cmd = [NVCC, *FLAGS, *(["-Xptxas", "-v"] if verbose else []), "-c", "-o", o + tag, s]
            jobs.append((subprocess.Popen(cmd), o))
    failed = [j.args for j, _ in jobs if j.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])
    for _, o in jobs:
        os.replace(o + tag, o)
    subprocess.run([NVCC, *FLAGS, "-shared", "-o", LIB + tag, *objects], check=True)
    os.replace(LIB + tag, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
