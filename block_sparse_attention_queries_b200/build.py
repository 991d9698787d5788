"""Builds libab.so (the CUDA library behind include/ab.h) for sm_100a and _marshal.so (the binding's checks of torch
tensors), in place."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC = os.path.join(HERE, "csrc", "ab_api.cu")
LIB = os.path.join(HERE, "libab.so")
MARSHAL_SRC = os.path.join(HERE, "csrc", "marshal.cpp")
MARSHAL = os.path.join(HERE, "_marshal.so")
HEADER = os.path.join(ROOT, "include", "ab.h")
DEPS = [os.path.join(HERE, "csrc", f) for f in sorted(os.listdir(os.path.join(HERE, "csrc")))
        if f != os.path.basename(MARSHAL_SRC)] + [HEADER]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-shared", "-Xcompiler", "-fPIC",
    "--expt-relaxed-constexpr",
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    raise RuntimeError("nvcc not found")


def _older(target: str, deps) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(p) > os.path.getmtime(target) for p in deps)


def needs_build() -> bool:
    return _older(LIB, DEPS)


def marshal_command() -> list:
    import torch
    base = os.path.dirname(torch.__file__)
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I", os.path.join(ROOT, "include"), "-isystem", os.path.join(base, "include"),
            "-isystem", sysconfig.get_paths()["include"], MARSHAL_SRC, "-L", os.path.join(base, "lib"), "-ltorch_python",
            "-ltorch_cpu", "-lc10", "-o", MARSHAL + ".tmp"]


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    jobs = []
    if force or needs_build():
        jobs.append(([nvcc(), *NVCC_FLAGS, *extra, "-I", os.path.join(ROOT, "include"), "-o", LIB + ".tmp", SRC], LIB))
    if force or _older(MARSHAL, [MARSHAL_SRC, HEADER]):
        jobs.append((marshal_command(), MARSHAL))
    running = []
    for cmd, target in jobs:
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        running.append((subprocess.Popen(cmd), cmd, target))
    for p, cmd, target in running:
        if p.wait() == 0:
            os.replace(target + ".tmp", target)
    for p, cmd, target in running:
        if p.returncode != 0:
            raise subprocess.CalledProcessError(p.returncode, cmd)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
