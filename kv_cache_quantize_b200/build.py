"""Build libkvq.so, the sm_100a CUDA library behind include/kvq.h, and _calls.so,
the extension module that passes torch tensors to its attention and page calls.

nvcc cross-compiles for sm_100a without a GPU.  -fmad=false keeps every
binary32 multiply and add separately rounded (the kernels also use the
explicitly rounded intrinsics); the CUDA runtime is linked statically so the
library only needs the driver.
"""
import importlib.metadata
import os
import re
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libkvq.so")
OBJ = os.path.join(HERE, "_build")
CALLS = os.path.join(HERE, "_calls.so")
CALLS_SOURCE = os.path.join(CSRC, "calls.cpp")
CALLS_TORCH = os.path.join(OBJ, "calls.torch")       # the torch and Python that _calls.so was built for
CXX = os.environ.get("CXX", "g++")
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


def installed_torch() -> str:
    return f"{importlib.metadata.version('torch')} {sys.implementation.cache_tag}"


def calls_torch() -> str:
    """What _calls.so was built for, or nothing where that is not known."""
    if not os.path.exists(CALLS_TORCH):
        return ""
    with open(CALLS_TORCH, encoding="utf-8") as f:
        return f.read()


def _calls_stale() -> bool:
    return _stale(CALLS, _deps(CALLS_SOURCE) | {os.path.abspath(__file__)}) or calls_torch() != installed_torch()


def needs_build() -> bool:
    return _stale(LIB, {os.path.abspath(__file__)}.union(*(_deps(s) for s in SOURCES))) or _calls_stale()


def _calls_command(out):
    import torch
    from torch.utils import cpp_extension
    cuda = os.path.join(os.path.dirname(os.path.dirname(shutil.which(NVCC) or "/usr/local/cuda/bin/nvcc")), "include")
    include = [sysconfig.get_paths()["include"], *cpp_extension.include_paths(), cuda, os.path.join(ROOT, "include")]
    return [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *("-isystem" + p for p in include), "-o", out, CALLS_SOURCE,
            "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
            "-L" + HERE, "-l:libkvq.so", "-Wl,-rpath,$ORIGIN"]


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
    if force or _calls_stale():
        subprocess.run(_calls_command(CALLS + tag), check=True)
        if os.path.exists(CALLS_TORCH):
            os.remove(CALLS_TORCH)             # a build that stops here is of unknown origin
        os.replace(CALLS + tag, CALLS)
        with open(CALLS_TORCH, "w", encoding="utf-8") as f:
            f.write(installed_torch())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
