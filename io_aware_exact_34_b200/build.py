"""Build ``libfattn.so`` in-tree with nvcc for sm_100a, and ``_fattn_calls.*.so``,
the native part of its Python binding, with g++ against the installed torch.

    python -m io_aware_exact_34_b200.build [--verbose]

The shared library links the CUDA runtime statically and resolves the
driver's tensor-map encoder at run time, so it loads on a machine without a
GPU (every entry point then reports FATTN_ERR_NO_DEVICE).  It needs neither
torch nor Python; where the native part of the binding cannot be built (no
torch, no headers of it or of Python), a warning says why and the binding goes
without it.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

from . import calls_path

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC = os.path.join(PKG, "csrc", "fattn_api.cu")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libfattn.so")
DEPS = [os.path.join(PKG, "csrc", f) for f in os.listdir(os.path.join(PKG, "csrc")) if f.endswith((".cu", ".cuh"))] + [
    os.path.join(INCLUDE, "fattn.h")]
CALLS_SRC = os.path.join(PKG, "csrc", "binding.cpp")


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in DEPS)


def build_calls(force: bool = False) -> str:
    """The binding's native calls (no CUDA code: any host compiler), for the installed torch."""
    try:
        import torch
    except ImportError as e:
        raise RuntimeError(f"torch does not import ({e})") from e
    out = calls_path(torch.__version__)
    if not force and os.path.exists(out) and os.path.getmtime(out) >= os.path.getmtime(CALLS_SRC):
        return out
    torch_dir = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    tmp = out + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared"]
    for d in (os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
              sysconfig.get_paths()["include"], os.path.join(cuda, "include")):
        cmd += ["-isystem", d]
    cmd += [CALLS_SRC, "-L", os.path.join(torch_dir, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed:\n" + res.stdout + res.stderr)
    os.replace(tmp, out)
    return out


def build(force: bool = False, verbose: bool = False) -> str:
    build_lib(force, verbose)
    try:
        build_calls(force)
    except (RuntimeError, OSError) as e:
        warnings.warn(f"the native calls of the Python binding are not built, it goes without them: {e}")
    return LIB


def build_lib(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [_nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
           "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC", "-shared", "-I", INCLUDE,
           "-o", tmp, SRC]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    if verbose:
        sys.stderr.write(res.stdout + res.stderr)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force=True, verbose="--verbose" in sys.argv)
    print(LIB)
