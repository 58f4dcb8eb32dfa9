"""In-tree build of the GEMV C-ABI library ``_lib/libgemv.so`` with nvcc.

Each translation unit is compiled for sm_103a in parallel, then linked into a
shared library with the CUDA runtime linked statically (so the library does
not depend on which libcudart the host process loaded).  The library knows
nothing of torch: Python calls it through ctypes, and for the operators of
gemv_ops.h through ``_lib/operators_py.so``, a small extension module that turns
torch tensors into pointers, sizes and strides (host code, built against the
installed torch and linked with the library).
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig
import threading
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(ROOT, "_build", "gemv")
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "libgemv.so")
HOST_TOOL_SRC = "bench_tool_main.cu"
HOST_TOOL = os.path.join(LIBDIR, "gemv_bench_tool")  # native host-overhead and read-ceiling measurements

EXTENSION_SRC = "operators_py.cpp"
EXTENSION = os.path.join(LIBDIR, "operators_py.so")

SOURCES = ["gemv_api.cu", "gemv_kernels_f16.cu", "gemv_kernels_bf16.cu", "gemv_bulk_f16.cu", "gemv_bulk_bf16.cu",
           "gla_decode.cu", "rms_norm.cu", "gated_scan.cu", "gemm.cu"]
HEADERS = [os.path.join(CSRC, h) for h in ("gemv_internal.h", "gemv_kernels.cuh", "gemv_tiles.cuh",
                                           "gemv_bulk.cuh", "ops_internal.h", "tc_ptx.cuh",
                                           "tensor_map.h")] + \
    [os.path.join(INCLUDE, h) for h in ("gemv.h", "gemv_ops.h")]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-I" + INCLUDE, "-I" + CSRC]

_lock = threading.Lock()


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the GEMV library needs the CUDA toolkit to build")
    return cand


def _stale() -> bool:
    products = (LIB, HOST_TOOL, EXTENSION)
    if not all(os.path.exists(f) for f in products):
        return True
    t = min(os.path.getmtime(f) for f in products)
    deps = [os.path.join(CSRC, s) for s in SOURCES + [HOST_TOOL_SRC, EXTENSION_SRC]] + HEADERS + [os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_dir() -> str:
    import torch
    return os.path.dirname(os.path.abspath(torch.__file__))


def _run(cmd, what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")


def _compile_extension() -> str:
    obj = os.path.join(OBJDIR, "operators_py.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-c", os.path.join(CSRC, EXTENSION_SRC), "-o", obj,
          "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(_torch_dir(), "include"), "-I" + cuda,
          "-I" + INCLUDE], f"g++ failed for {EXTENSION_SRC}")
    return obj


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile (if needed) and return the path of ``libgemv.so``."""
    with _lock:
        if not force and not _stale():
            return LIB
        os.makedirs(OBJDIR, exist_ok=True)
        os.makedirs(LIBDIR, exist_ok=True)
        exe = nvcc()

        def compile_one(src):
            obj = os.path.join(OBJDIR, os.path.splitext(src)[0] + ".o")
            cmd = [exe, *NVCC_FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
            if verbose and (r.stdout or r.stderr):
                print(r.stdout + r.stderr)
            return obj

        with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
            extension_obj = ex.submit(_compile_extension)
            objs = list(ex.map(compile_one, SOURCES))
            extension_obj = extension_obj.result()
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [exe, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-cudart", "static", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
        # the extension module and the native measurement tool, linked against the library just built
        tmp = EXTENSION + f".tmp{os.getpid()}"
        _run(["g++", "-shared", "-o", tmp, extension_obj, "-L" + LIBDIR, "-lgemv", "-Wl,-rpath,$ORIGIN",
              "-L" + os.path.join(_torch_dir(), "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"],
             "extension link failed")
        os.replace(tmp, EXTENSION)
        tmp = HOST_TOOL + f".tmp{os.getpid()}"
        cmd = [exe, *NVCC_FLAGS, *extra_flags, os.path.join(CSRC, HOST_TOOL_SRC), "-o", tmp,
               "-L" + LIBDIR, "-lgemv", "-Xlinker", "-rpath,$ORIGIN"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"measurement tool build failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, HOST_TOOL)
        return LIB


def ensure_built() -> str:
    return build(force=False)


def lib_path() -> str:
    return LIB
