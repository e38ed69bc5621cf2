"""Build libmla.so (the C-ABI decode library) for sm_103a with nvcc, and the
native part of the Python binding with g++.

Each translation unit is compiled in parallel, then linked into
``paged_mla_decode_07_gb300/_build/libmla.so`` and ``_mla_binding.*.so`` beside
it (in-tree, git-ignored).
Usage: ``python -m paged_mla_decode_07_gb300.builder [--verbose]``.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libmla.so")


def binding_path() -> str:
    """The binding's file.  It is compiled against the C++ types of one torch and the headers of one
    Python, which its name states: under others it is another file, not built yet."""
    abi = f"{sysconfig.get_config_var('SOABI')}.torch-{torch.__version__}-cxx11abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
    return os.path.join(BUILD, f"_mla_binding.{abi}.so")


BINDING = binding_path()
HEADER = os.path.join(HERE, "..", "include", "mla.h")
BINDING_SOURCE = "binding.cpp"
SOURCES = ["mla_api.cu", "mla_sched.cu", "mla_decode.cu", "mla_decode_pair.cu", "mla_combine.cu", "mla_noalloc.cu",
           "mla_store.cu", "mla_index.cu", "mla_pages.cu", "mla_prefix.cu", "mla_decode_rows.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libmla")
    return path


def _newer(target, *sources) -> bool:
    """target exists and is not older than its sources and this file."""
    return os.path.exists(target) and all(os.path.getmtime(f) <= os.path.getmtime(target)
                                          for f in (*sources, os.path.abspath(__file__)))


def library_up_to_date() -> bool:
    return _newer(LIB, HEADER, *(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != BINDING_SOURCE))


def binding_up_to_date() -> bool:
    return _newer(BINDING, HEADER, os.path.join(CSRC, BINDING_SOURCE))


def up_to_date() -> bool:
    return library_up_to_date() and binding_up_to_date()


def _run(what, cmd, verbose=False):
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:  # no such program
        raise RuntimeError(f"{what} failed: {e}") from e
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    if verbose:
        sys.stderr.write(r.stdout + r.stderr)


def build_library(verbose: bool = False) -> None:
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if verbose else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        _run(f"nvcc for {src}", [cc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj], verbose)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    _run("link", [cc, *ARCH, "-shared", "-o", tmp, *objs])
    os.replace(tmp, LIB)


def compile_binding() -> str:
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    obj = os.path.join(BUILD, "binding.o")
    _run(f"g++ for {BINDING_SOURCE}",
         ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          *(f"-isystem{p}" for p in (sysconfig.get_paths()["include"], inc,
                                     os.path.join(inc, "torch", "csrc", "api", "include"), cuda)),
          "-c", os.path.join(CSRC, BINDING_SOURCE), "-o", obj])
    return obj


def link_binding(obj: str) -> None:
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    _run("link of the binding",
         ["g++", "-shared", "-o", tmp, obj, f"-L{BUILD}", "-l:libmla.so", "-Wl,-rpath,$ORIGIN",
          f"-L{torch_lib}", f"-Wl,-rpath,{torch_lib}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"])
    os.replace(tmp, BINDING)


def build(force: bool = False, verbose: bool = False) -> str:
    """Build what is not up to date.  Without the library nothing works; without the binding, which
    needs g++ and the headers of Python and torch, the paged-cache calls go through ctypes."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        obj = ex.submit(compile_binding) if force or not binding_up_to_date() else None
        if force or not library_up_to_date():
            build_library(verbose)
        if obj is not None:
            try:
                link_binding(obj.result())
            except RuntimeError as e:
                warnings.warn(f"the native binding was not built; calls go through ctypes: {e}", RuntimeWarning, stacklevel=2)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose="--verbose" in sys.argv))
