"""Build libradattn.so in-tree: nvcc for sm_100a, static CUDA runtime.

    python static_sparse_attention_b200/build.py [--force] [--verbose] [--debug]

`--verbose` adds -Xptxas -v (registers, spills, shared memory per kernel).
`--debug` builds libradattn_debug.so instead: the same sources with
-DRA_DEBUG_BOUNDS, whose kernels check every global index and TMA coordinate
they derive from their inputs and record a failure in the device error word
(RA_ERR_DEVICE_BOUNDS) instead of making the access.  The binding loads it when
RA_LIBRARY_VARIANT=debug is set.

Where torch is installed both also build _torch_binding.so (g++, torch's headers), the
tensor checks of the operators whose calls last microseconds; it takes the entry points'
addresses from the package and is not linked to the library, which needs no torch.
"""
from __future__ import annotations

import glob
import hashlib
import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libradattn.so")
LIB_DEBUG = os.path.join(PKG, "libradattn_debug.so")

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC,-O3",
    "--cudart", "static",
    "-shared",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) \
        + glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(p) > t for p in deps)


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


BINDING_SRC = os.path.join(CSRC, "torch_binding.cpp")
BINDING = os.path.join(PKG, "_torch_binding.so")
BINDING_TORCH = os.path.join(PKG, "_build", "binding_torch")  # which torch it was built for


def _torch_folder() -> str | None:
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec else None


def _torch_version(torch: str) -> str:
    with open(os.path.join(torch, "version.py")) as fh:
        return hashlib.sha256(fh.read().encode()).hexdigest()


def _binding_stale(torch: str) -> bool:
    if not os.path.exists(BINDING) or not os.path.exists(BINDING_TORCH):
        return True
    with open(BINDING_TORCH) as fh:  # the extension fits one torch's headers
        if fh.read() != _torch_version(torch):
            return True
    return any(os.path.getmtime(p) > os.path.getmtime(BINDING) for p in (BINDING_SRC, os.path.join(INCLUDE, "radattn.h")))


def build_binding(force: bool = False) -> str | None:
    """The tensor side of the operators; None without torch (the library needs none)."""
    torch = _torch_folder()
    if torch is None:
        return None
    if not force and not _binding_stale(torch):
        return BINDING
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    tmp = BINDING + f".tmp{os.getpid()}"
    # the compiler on PATH, as nvcc's host compiler: one that links its own copy of
    # libstdc++ into the extension makes two in the process, and printing an error crash
    subprocess.check_call([
        "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", INCLUDE,
        "-I", os.path.join(torch, "include"), "-I", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
        "-I", sysconfig.get_path("include"), "-I", os.path.join(cuda, "include"), BINDING_SRC, "-o", tmp,
        "-L", os.path.join(torch, "lib"),
        *("-l" + lib for lib in ("torch_python", "torch", "torch_cpu", "torch_cuda", "c10", "c10_cuda"))])
    os.replace(tmp, BINDING)
    os.makedirs(os.path.dirname(BINDING_TORCH), exist_ok=True)
    with open(BINDING_TORCH, "w") as fh:
        fh.write(_torch_version(torch))
    return BINDING


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    lib = LIB_DEBUG if debug else LIB
    if not force and not _stale(lib):
        build_binding(force)
        return lib
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc(), *NVCC_FLAGS, *(["-DRA_DEBUG_BOUNDS"] if debug else []), "-I", INCLUDE, "-I", CSRC, *sources(),
           "-o", tmp]
    if verbose:
        cmd[1:1] = ["-Xptxas", "-v"]
    subprocess.check_call(cmd)
    os.replace(tmp, lib)
    build_binding(force)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv, debug="--debug" in sys.argv))
