"""Build the sm_100a shared library ``libpagedattn.so`` in-tree with nvcc.

Each translation unit is compiled to an object of its own, the units at the
same time, and only those whose sources or flags changed; then they are linked.
What a file was made with stands in a stamp beside its object."""

from __future__ import annotations

import contextlib
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor
from typing import Optional

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
NATIVE_FLAGS = ["-O2", "-std=c++17", "-fPIC"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: cannot build libpagedattn.so")
    return cand


def _headers() -> list:
    return sorted(glob.glob(os.path.join(ROOT, "include", "*.h")))


def sources() -> list:
    """What the library is made of."""
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  [u for u in UNITS if u.endswith(".cpp")]) + _headers()


def _newer(target: str, than: list) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(s) <= os.path.getmtime(target) for s in than)


def library_up_to_date() -> bool:
    return _newer(LIB, sources())


def native_up_to_date() -> bool:
    return _newer(NATIVE, [NATIVE_SRC, *_headers()]) and native_fits_torch()


def native_fits_torch() -> bool:
    """Whether the native module there is was built for the torch that is installed."""
    return _made_with(NATIVE) in (None, _native_key())


def _stamp(target: str) -> str:
    return os.path.join(OBJ_DIR, os.path.basename(target) + ".made")


def _made_with(target: str) -> Optional[str]:
    """What a file was made with; None where that is not known (it came without its objects)."""
    try:
        with open(_stamp(target)) as f:
            return f.read()
    except FileNotFoundError:
        return None


def _made(tmp: str, target: str, key: str) -> None:
    """A file is complete: it takes its place, with its stamp (none at all in between)."""
    with contextlib.suppress(FileNotFoundError):
        os.remove(_stamp(target))
    os.replace(tmp, target)
    with open(tmp + ".made", "w") as f:
        f.write(key)
    os.replace(tmp + ".made", _stamp(target))


def _library_key(extra_flags) -> str:
    return " ".join([*NVCC_FLAGS, *(extra_flags or [])])


def _native_key() -> str:
    import torch

    return " ".join([*NATIVE_FLAGS, "torch", torch.__version__, str(torch.compiled_with_cxx11_abi())])


def _object(unit: str) -> str:
    return os.path.join(OBJ_DIR, os.path.basename(unit) + ".o")


def _fresh(obj: str, key: str) -> bool:
    """Whether an object was made with these flags and is newer than every source its compiler read."""
    if not (os.path.exists(obj) and os.path.exists(obj + ".d")) or _made_with(obj) != key:
        return False
    with open(obj + ".d") as f:
        deps = f.read().replace("\\\n", " ").split(":", 1)[1].split()
    t = os.path.getmtime(obj)
    return all(os.path.exists(d) and os.path.getmtime(d) <= t for d in deps)


def _run(cmd: list, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)


def _compile(unit: str, force: bool, verbose: bool, extra_flags) -> str:
    obj, key = _object(unit), _library_key(extra_flags)
    if not force and _fresh(obj, key):
        return obj
    tmp = f"{obj}.tmp{os.getpid()}"
    cmd = [_nvcc(), *NVCC_FLAGS, *(extra_flags or []), "-I", os.path.join(ROOT, "include"), "-MMD", "-MF", tmp + ".d",
           "-c", "-o", tmp, unit]
    _run(cmd, verbose)
    os.replace(tmp + ".d", obj + ".d")
    _made(tmp, obj, key)
    return obj


def _torch_flags() -> tuple:
    """Include paths and link flags of the installed torch."""
    import torch
    from torch.utils import cpp_extension

    inc = [sysconfig.get_paths()["include"], *cpp_extension.include_paths(device_type="cuda")]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    abi = f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"
    return ([abi, *[x for d in inc for x in ("-isystem", d)]],
            ["-L" + lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"])


def _compile_native(force: bool, verbose: bool) -> str:
    obj, key = _object(NATIVE_SRC), _native_key()
    if not force and _fresh(obj, key):
        return obj
    tmp = f"{obj}.tmp{os.getpid()}"
    cmd = ["g++", *NATIVE_FLAGS, *_torch_flags()[0], "-MMD", "-MF", tmp + ".d", "-MT", "object", "-c",
           "-o", tmp, NATIVE_SRC]
    _run(cmd, verbose)
    os.replace(tmp + ".d", obj + ".d")
    _made(tmp, obj, key)
    return obj


def build_library(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """The library alone: nvcc is all it needs.  One that was made with other flags is made
    again (what opens the library takes it as it is, an instrumented one too)."""
    key = _library_key(extra_flags)
    if not force and library_up_to_date() and _made_with(LIB) in (None, key):
        return LIB
    os.makedirs(OBJ_DIR, exist_ok=True)
    with ThreadPoolExecutor(len(UNITS)) as pool:
        objs = list(pool.map(lambda u: _compile(u, force, verbose, extra_flags), UNITS))
    tmp = LIB + f".tmp{os.getpid()}"
    _run([_nvcc(), *NVCC_FLAGS, "-shared", "-o", tmp, *objs], verbose)
    _made(tmp, LIB, key)
    return LIB


def _link_native(obj: str, verbose: bool) -> str:
    tmp = NATIVE + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, "-L" + PKG, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN",
          *_torch_flags()[1]], verbose)
    _made(tmp, NATIVE, _native_key())
    return NATIVE


def build_native(force: bool = False, verbose: bool = False) -> str:
    """The Python entry of the per-step calls, which needs g++, the headers of
    torch and Python, and LIB, to which it is linked."""
    if not force and native_up_to_date():
        return NATIVE
    os.makedirs(OBJ_DIR, exist_ok=True)
    return _link_native(_compile_native(force, verbose), verbose)


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Both, compiled at the same time.  Where the native module cannot be built
    this raises, with the library in place."""
    os.makedirs(OBJ_DIR, exist_ok=True)
    with ThreadPoolExecutor(1) as pool:
        stale = force or not native_up_to_date()
        obj = pool.submit(_compile_native, force, verbose) if stale else None
        build_library(force, verbose, extra_flags)
        if obj is not None:
            _link_native(obj.result(), verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, extra_flags=["-Xptxas", "-v"] if "-v" in sys.argv else None)
    print(LIB)
