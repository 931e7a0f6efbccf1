"""Build libkvq.so (the C-ABI CUDA library) in-tree with nvcc for sm_103a, and
the native argument marshalling of the Python binding with g++."""
from __future__ import annotations

import glob
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libkvq.so")
# The same sources built with per-phase %globaltimer stamps in the decode and
# tag-check kernels (bench.py --phase-stamps); never the product library.
STAMPS_LIB = os.path.join(BUILD, "libkvq_stamps.so")

# Argument marshalling for the Python binding (csrc/kvq_binding.cpp): a CPython
# extension against the installed torch's headers; it calls libkvq through
# the entry points it is given and links none of it.
NATIVE = os.path.join(BUILD, "_kvq_native.so")
NATIVE_SRC = os.path.join(CSRC, "kvq_binding.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-I", INCLUDE,
]


def _nvcc() -> str:
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(cuda, "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + [NATIVE_SRC] + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) \
        + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def build_native() -> str:
    """Compile kvq_binding.cpp against the installed torch."""
    import sysconfig

    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    tmp = NATIVE + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", sysconfig.get_paths()["include"], "-isystem", inc, "-isystem", os.path.join(cuda, "include"),
           NATIVE_SRC, "-o", tmp, "-L", libs, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {NATIVE_SRC}:\n{r.stderr}")
    os.replace(tmp, NATIVE)
    return NATIVE


def build(force: bool = False, verbose: bool = False, stamps: bool = False) -> str:
    """Compile every .cu under csrc/ in parallel and link libkvq.so (with
    stamps=True: libkvq_stamps.so, the instrumented variant), and the native
    marshalling beside it."""
    lib = STAMPS_LIB if stamps else LIB
    objdir = os.path.join(BUILD, "stamps") if stamps else BUILD
    os.makedirs(objdir, exist_ok=True)
    if not force and os.path.exists(lib) and os.path.exists(NATIVE):
        newest = max(os.path.getmtime(p) for p in _deps())
        if min(os.path.getmtime(lib), os.path.getmtime(NATIVE)) >= newest:
            return lib
    nvcc = _nvcc()
    extra = ["-DKVQ_PHASE_STAMPS"] if stamps else []

    def compile_one(src):
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [nvcc] + NVCC_FLAGS + extra + ["-c", src, "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        return obj, r.stderr

    with ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        native = ex.submit(build_native)
        results = list(ex.map(compile_one, sources()))
        native.result()
    if verbose:
        for _, log in results:
            print(log)
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc, "-shared", "-gencode", "arch=compute_103a,code=sm_103a", "-o", tmp] + \
        [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
