"""Build the sm_100a shared library ``libpagedattn.so`` in-tree with nvcc.

Each translation unit is compiled to an object of its own, the units at the
same time, and only those whose sources changed; then they are linked."""

from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libpagedattn.so")
MAIN = os.path.join(CSRC, "pagedattn.cu")
# Translation units: the append, decode and prefill kernels and their C ABI,
# the drafting step's operators and theirs, and the host block manager.
UNITS = [MAIN, os.path.join(CSRC, "tree_ops.cu"), os.path.join(CSRC, "block_manager.cpp")]
OBJ_DIR = os.path.join(PKG, "_build")
# The Python entry of the per-step calls (host code, linked to torch and to LIB).
NATIVE_SRC = os.path.join(CSRC, "native_binding.cpp")
NATIVE = os.path.join(PKG, "_native" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))

NVCC_FLAGS = [
    "-gencode",
    "arch=compute_100a,code=sm_100a",
    "-lineinfo",
    "-O3",
    "-std=c++17",
    "-Xcompiler",
    "-fPIC",
]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: cannot build libpagedattn.so")
    return cand


def sources() -> list:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(os.path.join(ROOT, "include", "*.h")))


def up_to_date() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(NATIVE)):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(NATIVE))
    return all(os.path.getmtime(s) <= t for s in sources())


def _object(unit: str) -> str:
    return os.path.join(OBJ_DIR, os.path.basename(unit) + ".o")


def _fresh(obj: str) -> bool:
    """Whether an object is newer than every source its compiler read."""
    if not (os.path.exists(obj) and os.path.exists(obj + ".d")):
        return False
    with open(obj + ".d") as f:
        deps = f.read().replace("\\\n", " ").split(":", 1)[1].split()
    t = os.path.getmtime(obj)
    return all(os.path.exists(d) and os.path.getmtime(d) <= t for d in deps)


def _compile(unit: str, force: bool, verbose: bool, extra_flags) -> str:
    obj = _object(unit)
    if not force and _fresh(obj):
        return obj
    tmp = f"{obj}.tmp{os.getpid()}"
    cmd = [_nvcc(), *NVCC_FLAGS, *(extra_flags or []), "-I", os.path.join(ROOT, "include"), "-MMD", "-MF", tmp + ".d",
           "-c", "-o", tmp, unit]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp + ".d", obj + ".d")
    os.replace(tmp, obj)
    return obj


def _torch_flags() -> tuple:
    """Include paths and link flags of the installed torch."""
    import torch
    from torch.utils import cpp_extension

    inc = [sysconfig.get_paths()["include"], "/usr/local/cuda/include", *cpp_extension.include_paths()]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    abi = f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"
    return ([abi, *[x for d in inc for x in ("-isystem", d)]],
            ["-L" + lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"])


def _compile_native(force: bool, verbose: bool) -> str:
    obj = _object(NATIVE_SRC)
    if not force and _fresh(obj):
        return obj
    tmp = f"{obj}.tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", *_torch_flags()[0], "-MMD", "-MF", tmp + ".d", "-MT", "object", "-c",
           "-o", tmp, NATIVE_SRC]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp + ".d", obj + ".d")
    os.replace(tmp, obj)
    return obj


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJ_DIR, exist_ok=True)
    with ThreadPoolExecutor(len(UNITS) + 1) as pool:
        native = pool.submit(_compile_native, force, verbose)
        objs = list(pool.map(lambda u: _compile(u, force, verbose, extra_flags), UNITS))
        native = native.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [_nvcc(), *NVCC_FLAGS, "-shared", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    tmp = NATIVE + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, native, "-L" + PKG, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN",
           *_torch_flags()[1]]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, NATIVE)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, extra_flags=["-Xptxas", "-v"] if "-v" in sys.argv else None)
    print(LIB)
