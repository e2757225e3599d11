"""Build the CUDA library (libdsa.so) in-tree with nvcc for sm_100a.

The library is the C ABI declared in include/dsa.h; the Python binding loads
it with ctypes.  Run ``python -m dynamic_block_sparse_dsa_b200.build``.
"""
from __future__ import annotations

import glob
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libdsa.so")
ARGS_SRC = os.path.join(CSRC, "tensor_args.cpp")
ARGS_LIB = os.path.join(PKG, "_tensor_args" + sysconfig.get_config_var("EXT_SUFFIX"))   # for this Python alone
HEADER = os.path.join(ROOT, "include", "dsa.h")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libdsa.so")


def sources() -> list:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs() -> list:
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))) + \
        [HEADER, os.path.abspath(__file__)]


def is_stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in _inputs())


def _args_command() -> list:
    """The compiler and its arguments, without the output, for the reader of tensor arguments."""
    import torch
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"]]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[a for i in inc for a in ("-isystem", i)], ARGS_SRC, "-L" + os.path.join(root, "lib"), "-ltorch_python",
            "-ltorch_cpu", "-lc10"]


def args_key() -> str:
    """Names what the reader is built from: its source, the structs that it fills, the command, torch and Python."""
    import torch
    h = hashlib.sha256(repr((_args_command(), torch.__version__, torch.version.git_version, sys.version)).encode())
    for path in (ARGS_SRC, HEADER):
        with open(path, "rb") as f:
            h.update(f.read())
    return h.hexdigest()[:32]


def args_stale() -> bool:
    """Whether the reader is missing or built from anything else than what is here."""
    try:
        with open(ARGS_LIB + ".key") as f:
            return not os.path.exists(ARGS_LIB) or f.read() != args_key()
    except OSError:
        return True


def build_tensor_args(force: bool = False) -> bool:
    """Compile the binding's native tensor reader beside libdsa.so.  The binding
    does the same in Python without it, so a failure here is only reported."""
    if not force and not args_stale():
        return True
    tmp = ARGS_LIB + f".tmp{os.getpid()}"
    try:
        key = args_key()
        r = subprocess.run([*_args_command(), f'-DDSA_ARGS_KEY="{key}"', "-o", tmp], capture_output=True, text=True)
    except OSError as e:
        sys.stderr.write(f"tensor_args.cpp not built: {e}\n")
        return False
    if r.returncode != 0:
        sys.stderr.write(f"tensor_args.cpp not built ({r.returncode}):\n{r.stderr[-2000:]}\n")
        return False
    try:   # no key stands beside a reader that it does not belong to
        os.remove(ARGS_LIB + ".key")
    except OSError:
        pass
    os.replace(tmp, ARGS_LIB)
    with open(tmp, "w") as f:
        f.write(key)
    os.replace(tmp, ARGS_LIB + ".key")
    return True


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every csrc/*.cu into one shared library (static cudart), and the
    binding's tensor reader."""
    build_tensor_args(force)
    if not force and not is_stale():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc_path(), "-O3", "-std=c++17", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC", "-shared",
           "-I", os.path.join(ROOT, "include"), "-o", tmp, *sources()]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed ({r.returncode}):\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    if verbose:
        sys.stderr.write(r.stdout + r.stderr)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
