"""Build ``libgdn.so`` (the C-ABI CUDA library) in-tree with nvcc for sm_100a, and, where
PyTorch is installed, ``_gdn_torch.so`` (the binding's argument checks, host code against
PyTorch's headers).

Usage: ``python -m linear_attention_12_b200.build [--force] [--verbose]``.
The library is written next to this file so that it travels with the
repository snapshot; nothing is installed into site-packages.
"""
from __future__ import annotations

import argparse
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libgdn.so")
BINDING = os.path.join(HERE, "_gdn_torch.so")
BINDING_SRC = os.path.join(CSRC, "gdn_torch.cpp")
BUILD_DIR = os.path.join(HERE, "_build")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    deps.append(os.path.join(ROOT, "include", "gdn.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_version():
    """The installed PyTorch's version, or None."""
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return "unknown" if importlib.util.find_spec("torch") else None


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """Compile ``csrc/gdn_torch.cpp`` into ``_gdn_torch.so``; return its path."""
    deps = (BINDING_SRC, os.path.join(ROOT, "include", "gdn.h"))
    # (it fits the PyTorch and the Python it was compiled against)
    against = f"torch {_torch_version()}, {sysconfig.get_config_var('SOABI')}\n"
    stamp = os.path.join(BUILD_DIR, "_gdn_torch.txt")
    if (not force and os.path.exists(BINDING)
            and all(os.path.getmtime(d) <= os.path.getmtime(BINDING) for d in deps)
            and os.path.exists(stamp) and open(stamp).read() == against):
        return BINDING
    import torch
    t = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for d in (os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
              os.path.join(cuda, "include"), sysconfig.get_paths()["include"]):
        cmd += ["-I", d]
    cmd += [BINDING_SRC, "-o", tmp, "-L", os.path.join(t, "lib"), "-ltorch_python", "-ltorch_cuda",
            "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(tmp, BINDING)
    os.makedirs(BUILD_DIR, exist_ok=True)
    with open(stamp, "w") as f:
        f.write(against)
    return BINDING


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile every ``csrc/*.cu`` into ``libgdn.so``, then the binding's ``_gdn_torch.so``
    (where there is a PyTorch for it); return the library's path."""
    lib = build_library(force=force, verbose=verbose, ptxas_info=ptxas_info)
    if _torch_version() is None:
        print("no PyTorch: built the C library without _gdn_torch.so", file=sys.stderr)
        return lib
    try:
        build_binding(force=force, verbose=verbose)
    except Exception as e:
        raise RuntimeError(f"{lib} is built, but the Python binding's _gdn_torch.so could not be "
                           f"compiled: {e}") from e
    return lib


def build_library(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile every ``csrc/*.cu`` into ``libgdn.so``; return its path."""
    if not force and not _stale():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
                     "-rdc=true", "-I", os.path.join(ROOT, "include")]
    if ptxas_info:
        common += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc] + common + ["-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        subprocess.check_call(cmd)
        return obj

    with ThreadPoolExecutor(os.cpu_count() or 1) as pool:
        objs = list(pool.map(compile_one, sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc] + ARCH + ["-shared", "-Xcompiler", "-fPIC", "-o", tmp] + objs + ["-cudart", "static"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose, ptxas_info=a.ptxas_info))
