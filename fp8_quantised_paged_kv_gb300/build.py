"""Build libkvq.so (the C-ABI CUDA library) in-tree with nvcc for sm_103a, and
the native argument marshalling of the Python binding with g++.

The library needs nvcc alone (``python -m fp8_quantised_paged_kv_gb300.build
--library`` builds nothing else); the marshalling needs the installed torch's
headers, and is left out where there is no torch to marshal for."""
from __future__ import annotations

import glob
import importlib.metadata
import os
import subprocess
import sysconfig
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


def _newest(paths):
    return max(os.path.getmtime(p) for p in paths)


def _headers(*suffixes):
    return [h for s in suffixes for h in glob.glob(os.path.join(CSRC, s))] + glob.glob(os.path.join(INCLUDE, "*.h"))


def _current(target, deps) -> bool:
    return os.path.exists(target) and os.path.getmtime(target) >= _newest(deps + [os.path.abspath(__file__)])


def torch_version():
    """The installed torch's version (where its metadata say so without importing
    it), or None."""
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        pass
    try:
        import torch
    except ImportError:
        return None
    return torch.__version__


def native_path():
    """Where the marshalling for this torch and this Python lies, or None without
    torch.  Both are in the name: an extension built against another torch's
    C++ headers must not be loaded."""
    version = torch_version()
    if version is None:
        return None
    abi = sysconfig.get_config_var("SOABI") or "unknown"
    return os.path.join(BUILD, f"_kvq_native.torch-{version}.{abi}.so")


def build_native(force: bool = False) -> str:
    """Compile kvq_binding.cpp against the installed torch, if that is not done."""
    native = native_path()
    if native is None:
        raise RuntimeError("the Python binding needs torch, which is not installed")
    if not force and _current(native, [NATIVE_SRC] + glob.glob(os.path.join(INCLUDE, "*.h"))):
        return native
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    os.makedirs(BUILD, exist_ok=True)
    tmp = native + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", sysconfig.get_paths()["include"], "-isystem", inc, "-isystem", os.path.join(cuda, "include"),
           NATIVE_SRC, "-o", tmp, "-L", libs, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {NATIVE_SRC}:\n{r.stderr}")
    os.replace(tmp, native)
    return native


def build(force: bool = False, verbose: bool = False, stamps: bool = False, native: bool = True) -> str:
    """Compile every .cu under csrc/ in parallel and link libkvq.so (with
    stamps=True: libkvq_stamps.so, the instrumented variant); with native, and
    where torch is installed, the marshalling beside it.  The library is in
    place before a failure of the marshalling is raised."""
    lib = STAMPS_LIB if stamps else LIB
    objdir = os.path.join(BUILD, "stamps") if stamps else BUILD
    os.makedirs(objdir, exist_ok=True)
    with ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        binding = ex.submit(build_native, force) if native and torch_version() is not None else None
        if force or not _current(lib, sources() + _headers("*.h", "*.cuh")):
            _build_library(ex, lib, objdir, verbose, ["-DKVQ_PHASE_STAMPS"] if stamps else [])
        if binding is not None:
            binding.result()
    return lib


def _build_library(ex, lib: str, objdir: str, verbose: bool, extra: list) -> None:
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [nvcc] + NVCC_FLAGS + extra + ["-c", src, "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        return obj, r.stderr

    results = list(ex.map(compile_one, sources()))
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


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, native="--library" not in sys.argv))
