"""Builds the CUDA library librtlynx.so in-tree for sm_100a (nvcc, no GPU needed),
and, where torch is installed, the host code of its torch-level calls (g++).

    python -m activation_sparse_gemm_b200.build [--force] [--verbose-ptxas]
"""
from __future__ import annotations

import argparse
import glob
import importlib.util
import os
import runpy
import shutil
import subprocess
import sys
import sysconfig

from . import torch_lib_path

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIB_DIR, "librtlynx.so")
TORCH_SRC = os.path.join(CSRC, "torch_calls.cpp")
HEADER = os.path.join(ROOT, "include", "rtlynx.h")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def host_compiler() -> str:
    """The system's g++: the extension has to share torch's libstdc++, which a toolchain of its own may link statically."""
    for cand in ("/usr/bin/g++", shutil.which("g++")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("g++ not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))
    return any(os.path.getmtime(p) > t for p in deps)


def torch_dir():
    """Where torch is installed, or None."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec else None


def build_torch_calls(force: bool = False):
    """Compiles the torch-level calls against the installed torch (g++, about 20 s); None where there is no torch."""
    at = torch_dir()
    if at is None:
        return None
    out = torch_lib_path(runpy.run_path(os.path.join(at, "version.py"))["__version__"])
    if not force and os.path.exists(out) and \
            os.path.getmtime(out) >= max(os.path.getmtime(TORCH_SRC), os.path.getmtime(HEADER)):
        return out
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    os.makedirs(LIB_DIR, exist_ok=True)
    tmp = out + f".{os.getpid()}.tmp"
    subprocess.check_call([
        host_compiler(), "-O2", "-std=c++17", "-fPIC", "-shared",
        "-DTORCH_EXTENSION_NAME=rtlynx_torch", "-I" + sysconfig.get_paths()["include"],
        "-I" + os.path.join(at, "include"),
        "-I" + os.path.join(at, "include", "torch", "csrc", "api", "include"),
        "-I" + os.path.join(cuda, "include"), TORCH_SRC, "-o", tmp, "-L" + os.path.join(at, "lib"), "-lc10",
        "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_python"])
    os.replace(tmp, out)
    return out


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    build_library(force, verbose_ptxas)
    if build_torch_calls(force) is None:
        print("torch is not installed: librtlynx.so alone, without the torch-level calls", file=sys.stderr)
    return LIB


def build_library(force: bool = False, verbose_ptxas: bool = False) -> str:
    if not force and not needs_build():
        return LIB
    os.makedirs(LIB_DIR, exist_ok=True)
    obj_dir = os.path.join(LIB_DIR, "obj")
    os.makedirs(obj_dir, exist_ok=True)
    common = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "-I", os.path.join(ROOT, "include")]
    if verbose_ptxas:
        common += ["-Xptxas", "-v"]
    objs = []
    for src in sources():
        obj = os.path.join(obj_dir, os.path.basename(src) + ".o")
        subprocess.check_call(common + ["-c", src, "-o", obj])
        objs.append(obj)
    tmp = LIB + f".{os.getpid()}.tmp"
    subprocess.check_call([nvcc(), *ARCH, "-shared", "-o", tmp, *objs])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose_ptxas=a.verbose_ptxas))
    sys.exit(0)
