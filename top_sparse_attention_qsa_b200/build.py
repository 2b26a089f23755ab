"""Builds the libraries in-tree, with nvcc (sm_100a) and, for the binding, g++:

    libqsa.so        the kernels and the C ABI of include/qsa.h (production)
    libqsa_debug.so  measurement kernels and test hooks of include/qsa_debug.h,
                     compiled with QSA_DEBUG (the tests and the benchmark load
                     it next to libqsa.so; nothing in libqsa.so needs it)
    _binding.so      the CPython binding of the calls whose marshalling counts
                     (csrc/qsa_binding.cpp; against torch and libqsa.so)

    python -m top_sparse_attention_qsa_b200.build [--verbose] [--no-binding]

Both link the CUDA runtime statically and resolve the driver at run time, so
they load on machines without a GPU (their entry points then return
QSA_ERR_CUDA).
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libqsa.so")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_ABI = BINDING + ".abi"
DEBUG_LIB = os.path.join(PKG, "libqsa_debug.so")
DEBUG_SOURCES = ("qsa_debug_api.cu",)

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
    "--expt-relaxed-constexpr",
    "-cudart", "static",
]


def _sources(debug: bool = False):
    every = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    if debug:
        return [f for f in every if os.path.basename(f) in DEBUG_SOURCES]
    return [f for f in every if os.path.basename(f) not in DEBUG_SOURCES]


def _deps():
    return (sorted(glob.glob(os.path.join(CSRC, "*.cu"))) + glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(d) <= t for d in _deps())


def nvcc() -> str:
    cand = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    p = os.path.join(cand, "bin", "nvcc")
    return p if os.path.exists(p) else "nvcc"


def _build_one(lib: str, debug: bool, force: bool, verbose: bool) -> str:
    if not force and up_to_date(lib):
        return lib
    tmp = lib + f".tmp{os.getpid()}"
    extra = ["-DQSA_DEBUG"] if debug else []
    cmd = [nvcc()] + NVCC_FLAGS + extra + ["-I", INCLUDE, "-I", CSRC, "-shared", "-o", tmp] + _sources(debug)
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)
    if verbose:
        sys.stdout.write(res.stdout + res.stderr)
    os.replace(tmp, lib)
    return lib


def binding_abi() -> str:
    """The torch and the Python that a _binding.so built now belongs to (written beside it)."""
    import torch
    return (f"torch {torch.__version__}, cxx11 abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, "
            f"{sysconfig.get_config_var('SOABI')}\n")


def binding_up_to_date() -> bool:
    if not up_to_date(BINDING) or os.path.getmtime(BINDING) < os.path.getmtime(LIB) or not os.path.exists(BINDING_ABI):
        return False
    with open(BINDING_ABI) as f:
        return f.read() == binding_abi()


def _build_binding(force: bool) -> None:
    if not force and binding_up_to_date():
        return
    import torch
    base = os.path.dirname(torch.__file__)
    lib = os.path.join(base, "lib")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    tmp = BINDING + f".tmp{os.getpid()}"
    inc = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(base, "include"),
           os.path.join(base, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    cmd = (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
           + [x for i in inc for x in ("-isystem", i)] + [os.path.join(CSRC, "qsa_binding.cpp"), "-o", tmp, "-L", lib,
           "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", "-L", PKG, "-l:libqsa.so",
           "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib])
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)
    if os.path.exists(BINDING_ABI):
        os.remove(BINDING_ABI)                           # (it belongs to the binding that goes)
    os.replace(tmp, BINDING)
    with open(BINDING_ABI, "w") as f:
        f.write(binding_abi())


def build(force: bool = False, verbose: bool = False, debug: bool = True, binding: bool = True) -> str:
    """Builds libqsa.so, (debug=True) libqsa_debug.so and (binding=True) _binding.so; returns libqsa.so's path.
    The binding comes last: where it cannot be built (no torch, no Python headers), the error leaves the
    libraries in place, and with them every call but the cache appends and the 4-bit attention."""
    _build_one(LIB, False, force, verbose)
    if debug:
        _build_one(DEBUG_LIB, True, force, verbose)
    if binding:
        _build_binding(force)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose="--verbose" in sys.argv, binding="--no-binding" not in sys.argv))
