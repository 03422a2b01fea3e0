"""Build the CUDA library in-tree: block_scaled_fp8_persistent_gb300/lib/libbsfp8.so.

Each translation unit is compiled for sm_103a only (nvcc -gencode
arch=compute_103a,code=sm_103a), in parallel, then linked into one shared library with
the CUDA runtime linked statically (the driver itself is found at run time).

build(debug=True) makes lib/libbsfp8_debug.so instead: the same sources with
-DBSFP8_DEBUG=1, whose kernels check every tile's coordinates against the problem and
record BSFP8_ERR_DEVICE_BOUNDS in the device error word instead of going out of range.

Both also make lib/bsfp8_binding_<torch version>.so (csrc/binding.cpp, host code only): the
Python side of the operators around the GEMM, compiled against the torch that is installed.  The
library does not depend on it: where it cannot be built (no torch, no C++ compiler) there is a
warning, and only the Python calls of those operators are missing.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(PKG, "_build")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libbsfp8.so")
DEBUG_LIB = os.path.join(LIBDIR, "libbsfp8_debug.so")

SOURCES = ["capi.cu", "bsfp8_grouped.cu", "bsmxfp8_grouped.cu", "bsmxfp8_pair.cu",
           "capi_moe.cu", "moe_quant.cu", "moe_route.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + CSRC, "-I" + INCLUDE]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _deps() -> list[str]:
    out = [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    out += [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    return out


def binding_path() -> str:
    """The compiled binding of the torch that is installed."""
    from importlib.metadata import version
    v = "".join(c if c.isalnum() else "_" for c in version("torch"))
    return os.path.join(LIBDIR, f"bsfp8_binding_{v}.so")


def build_binding(force: bool = False) -> str:
    """Builds the compiled binding (raises if that fails)."""
    out = binding_path()
    if not force and up_to_date(out):
        return out
    from importlib.util import find_spec
    torch = os.path.dirname(find_spec("torch").origin)
    lib = os.path.join(torch, "lib")
    os.makedirs(LIBDIR, exist_ok=True)
    tmp = out + f".tmp{os.getpid()}"
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I" + INCLUDE, "-isystem", cuda,
           "-isystem", os.path.join(torch, "include"),
           "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], os.path.join(CSRC, "binding.cpp"),
           "-o", tmp, "-L" + lib, "-Wl,-rpath," + lib, "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)
    return out


def _try_binding(force: bool = False) -> None:
    try:
        build_binding(force)
    except Exception as e:  # whatever is missing: the library does not need it
        warnings.warn(f"the compiled binding was not built: {e}", RuntimeWarning, stacklevel=3)


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(d) <= t for d in _deps())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False,
          debug: bool = False) -> str:
    lib = DEBUG_LIB if debug else LIB
    objdir = OBJDIR + ("_debug" if debug else "")
    if not force and up_to_date(lib):
        _try_binding()
        return lib
    os.makedirs(objdir, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    if debug:
        extra.append("-DBSFP8_DEBUG=1")

    def compile_one(src: str) -> str:
        obj = os.path.join(objdir, src.replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_try_binding, force)
        objs = list(ex.map(compile_one, SOURCES))
        binding.result()
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, ptxas_info="-v" in sys.argv,
                debug="--debug" in sys.argv))
