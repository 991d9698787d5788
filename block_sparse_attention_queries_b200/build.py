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


def torch_version() -> str | None:
    """None: without torch, which only the binding needs."""
    try:
        import torch
    except ImportError:
        return None
    return torch.__version__


def needs_marshal() -> bool:
    """_marshal.so is missing, older than its source, or made for another torch (whose tensors it would misread)."""
    if _older(MARSHAL, [MARSHAL_SRC, HEADER]):
        return True
    with open(MARSHAL, "rb") as f:
        return f"AB_TORCH={torch_version()};".encode() not in f.read()


def marshal_command() -> list:
    import torch
    base = os.path.dirname(torch.__file__)
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            f'-DAB_TORCH="{torch.__version__}"',
            "-I", os.path.join(ROOT, "include"), "-isystem", os.path.join(base, "include"),
            "-isystem", sysconfig.get_paths()["include"], MARSHAL_SRC, "-L", os.path.join(base, "lib"), "-ltorch_python",
            "-ltorch_cpu", "-lc10", "-o", MARSHAL + ".tmp"]


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Brings both libraries up to date; without torch libab.so alone.  What can be built is, whatever fails."""
    running, errors = [], []

    def start(cmd, target):
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        try:
            running.append((subprocess.Popen(cmd), cmd, target))
        except OSError as e:
            errors.append(e)

    if force or needs_build():
        start([nvcc(), *NVCC_FLAGS, *extra, "-I", os.path.join(ROOT, "include"), "-o", LIB + ".tmp", SRC], LIB)
    if torch_version() is not None and (force or needs_marshal()):
        start(marshal_command(), MARSHAL)
    for p, cmd, target in running:
        if p.wait() == 0:
            os.replace(target + ".tmp", target)
        else:
            errors.append(subprocess.CalledProcessError(p.returncode, cmd))
    if errors:
        raise errors[0]
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
