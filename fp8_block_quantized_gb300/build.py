"""In-tree build of the jet_fp8 shared library for sm_103a.

Each ``csrc/*.cu`` is compiled to an object in parallel with
``nvcc -gencode arch=compute_103a,code=sm_103a -lineinfo -O3`` and the objects
are linked into ``_build/libjetfp8.so`` (CUDA runtime linked statically).
``pysrc/marshal.cpp``, the compiled part of the Python binding, becomes
``_build/_marshal-*.so`` (g++ against the installed torch's headers; it calls
the library through addresses the binding gives it).  The library needs nvcc
alone: where the module cannot be built, only the operators it marshals fail.
IEEE division and denormals are kept (no fast-math): the quantizers' codes must
be bit-exact.
"""
from __future__ import annotations

import glob
import importlib.metadata
import os
import shutil
import subprocess
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libjetfp8.so")
MARSHAL_SRC = os.path.join(PKG, "pysrc", "marshal.cpp")


def _marshal_name() -> str:
    """Of the module for this torch and this Python, whose binary interfaces it holds."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "none"
    return f"_marshal-torch{version}{sysconfig.get_config_var('EXT_SUFFIX')}"


MARSHAL = os.path.join(BUILD, _marshal_name())
INCLUDE = os.path.join(os.path.dirname(PKG), "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVFLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
                  "-ftz=false", "-prec-div=true", "-prec-sqrt=true",
                  "--expt-relaxed-constexpr", "-I", INCLUDE]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the jet_fp8 CUDA library cannot be built")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def _newer(out, deps) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(p) <= os.path.getmtime(out) for p in deps)


def up_to_date() -> bool:
    """Whether the library is (the binding's extension module apart)."""
    return _newer(LIB, _deps())


def marshal_up_to_date() -> bool:
    return _newer(MARSHAL, [MARSHAL_SRC, os.path.join(INCLUDE, "jet_fp8.h"), os.path.abspath(__file__)])


def build_marshal(force: bool = False) -> str:
    """Compile the binding's extension module against the installed torch; returns its path."""
    if not force and marshal_up_to_date():
        return MARSHAL
    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    os.makedirs(BUILD, exist_ok=True)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = MARSHAL + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++20", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-I", os.path.join(root, "include"),
           "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-I", os.path.join(cuda, "include"), MARSHAL_SRC, "-o", tmp,
           "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           f"-Wl,-rpath,{os.path.join(root, 'lib')}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for marshal.cpp:\n{r.stderr}")
    os.replace(tmp, MARSHAL)
    return MARSHAL


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link the library, and beside it the binding's extension module;
    returns the library's path.  A module that cannot be built is a warning."""
    with ThreadPoolExecutor(1) as beside:
        marshal = beside.submit(build_marshal, force)
        path = LIB if not force and up_to_date() else _build_library(verbose, extra_flags)
    if marshal.exception():
        warnings.warn(f"the binding's extension module is not built: {marshal.exception()}")
    return path


def _build_library(verbose, extra_flags) -> str:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    srcs = sources()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *NVFLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    with ThreadPoolExecutor(max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
