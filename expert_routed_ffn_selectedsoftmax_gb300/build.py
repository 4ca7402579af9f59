"""Compile the CUDA library (csrc/*.cu) into libmoe_gb300.so, in-tree, and the
Python module of the operators beside the layer (csrc/*_binding.cpp) into
_fp8b.<PyTorch's and Python's versions>.so beside it (binding_path()).

nvcc, one -gencode for sm_103a, translation units compiled in parallel (the
module by the host compiler against PyTorch's headers), no cmake.  Rebuilds only
when a source or header is newer than what was built.

The library is all that the C ABI needs.  Where the module cannot be built (no
PyTorch or Python headers), build() says so in a warning and the library stands;
only the calls that go through the module need it, and they raise without it.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG, "libmoe_gb300.so")
# the debug build (MOE_DEBUG=1: device-side checks of the grouping the expert
# kernels are given, include/moe_debug.h)
DEBUG_BUILD_DIR = os.path.join(ROOT, "_build_debug")
DEBUG_LIB_PATH = os.path.join(PKG, "libmoe_gb300_debug.so")

# the Python module of the operators beside the layer (block-scaled fp8, int8, dispatch and combine)
BINDING_SRCS = [os.path.join(CSRC, name) for name in ("fp8b_binding.cpp", "i8_binding.cpp")]
BINDING_HEADER = os.path.join(CSRC, "binding.h")


def binding_path() -> str:
    """Where the module of this interpreter and PyTorch lies.  It is bound to both
    (C++ classes, CPython's own ABI), so their versions are part of its name: after
    an upgrade, or from another environment on the same tree, an older build is not
    found instead of being loaded."""
    import torch
    tag = f"torch{torch.__version__}.cxx11abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
    return os.path.join(PKG, f"_fp8b.{tag}{sysconfig.get_config_var('EXT_SUFFIX')}")


ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden"] + ARCH


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoe_gb300.so")
    return cand


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")) + \
        [os.path.abspath(__file__)]


def _newer(path: str, deps) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path) for p in deps)


def up_to_date(lib: str = LIB_PATH) -> bool:
    return _newer(lib, _deps())


def binding_up_to_date() -> bool:
    return _newer(binding_path(), [*BINDING_SRCS, BINDING_HEADER, os.path.join(INCLUDE, "moe.h"), os.path.abspath(__file__)])


def _compile_binding(build_dir: str) -> list:
    """csrc/*_binding.cpp -> object files (host compiler, PyTorch's headers)."""
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda_inc = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    os.makedirs(build_dir, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(build_dir, os.path.basename(src)[:-4] + ".o")
        cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
               "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
               "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda_inc,
               "-I", INCLUDE, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{cmd[0]} failed on {os.path.basename(src)}:\n{r.stderr}")
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(BINDING_SRCS)) as ex:
        return list(ex.map(compile_one, BINDING_SRCS))


def _link_binding(objs: list) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    path = binding_path()
    tmp = path + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, *objs, "-L", PKG, "-l:" + os.path.basename(LIB_PATH),
           "-L", lib, "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-lc10", "-lc10_cuda",
           "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking {os.path.basename(path)} failed:\n{r.stderr}")
    os.replace(tmp, path)


def build(force: bool = False, verbose: bool = False, extra_flags=(), debug: bool = False) -> str:
    """Compile libmoe_gb300.so (or, with debug=True, libmoe_gb300_debug.so with
    MOE_DEBUG=1) from csrc/, and the module beside the former; returns the
    library's path.  Raises where the library cannot be built; warns where the
    module cannot (build_binding() raises)."""
    if debug:
        return _build_library(force, verbose, extra_flags, debug)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        objs = ex.submit(lambda: _compile_binding(BUILD_DIR) if force or not binding_up_to_date() else None)
        lib = _build_library(force, verbose, extra_flags, debug)
        try:
            if objs.result():
                _link_binding(objs.result())
        except Exception as e:   # (no PyTorch, no headers, no host compiler)
            _remove_stale()
            warnings.warn(f"the Python module of the operators beside the layer (_fp8b) was not built, their calls will raise: {e}",
                          RuntimeWarning, stacklevel=2)
    return lib


def _remove_stale() -> None:
    """A module of older sources is not to be loaded beside a newer library."""
    try:
        os.remove(binding_path())
    except (ImportError, OSError):
        pass


def build_binding(force: bool = False) -> str:
    """Compile the module if it is stale (the library has to be there); returns its path."""
    if force or not binding_up_to_date():
        _link_binding(_compile_binding(BUILD_DIR))
    return binding_path()


def _build_library(force, verbose, extra_flags, debug) -> str:
    lib = DEBUG_LIB_PATH if debug else LIB_PATH
    build_dir = DEBUG_BUILD_DIR if debug else BUILD_DIR
    if debug:
        extra_flags = (*extra_flags, "-DMOE_DEBUG=1")
    if not force and up_to_date(lib):
        return lib
    nvcc = _nvcc()
    os.makedirs(build_dir, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *NVCC_FLAGS, *extra_flags, "-I", INCLUDE, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True, debug="--debug" in sys.argv))
