"""In-tree build of the GEMV C-ABI library ``_lib/libgemv.so`` with nvcc.

Each translation unit is compiled for sm_103a in parallel, then linked into a
shared library with the CUDA runtime linked statically (so the library does
not depend on which libcudart the host process loaded).  The library knows
nothing of torch: Python calls it through ctypes, and for the operators of
gemv_ops.h through ``_lib/operators_py.so``, a small extension module that turns
torch tensors into pointers, sizes and strides (host code, built against the
installed torch and linked with the library).

Run as a script, this file builds the library and the measurement tool alone,
without torch or Python's headers.
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
EXTENSION_STAMP = os.path.join(LIBDIR, "operators_py.built")  # what it was built against

SOURCES = ["gemv_api.cu", "gemv_kernels_f16.cu", "gemv_kernels_bf16.cu", "gemv_bulk_f16.cu", "gemv_bulk_bf16.cu",
           "gla_decode.cu", "rms_norm.cu", "gated_scan.cu", "gemm.cu", "layer_norm.cu", "gated_delta.cu",
           "gated_delta_chunks_f16.cu", "gated_delta_chunks_bf16.cu", "gated_delta_gradient.cu",
           "gated_delta_tensor.cu"]
HEADERS = [os.path.join(CSRC, h) for h in ("gemv_internal.h", "gemv_kernels.cuh", "gemv_tiles.cuh",
                                           "gemv_bulk.cuh", "ops_internal.h", "tc_ptx.cuh",
                                           "tensor_map.h", "gated_delta.h", "gated_delta_mma.cuh",
                                           "gated_delta_chunks.cuh")] + \
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


def _older(products, sources) -> bool:
    """Whether a product is missing or older than one of the sources."""
    if not all(os.path.exists(f) for f in products):
        return True
    t = min(os.path.getmtime(f) for f in products)
    return any(os.path.getmtime(d) > t for d in sources)


def _stale_library() -> bool:
    deps = [os.path.join(CSRC, s) for s in SOURCES + [HOST_TOOL_SRC]] + HEADERS + [os.path.abspath(__file__)]
    return _older((LIB, HOST_TOOL), deps)


def _extension_target() -> str:
    """What the extension module's binary interface depends on."""
    import torch
    return f"torch {torch.__version__} python {sysconfig.get_config_var('SOABI')}"


def _stale_extension() -> bool:
    header = os.path.join(INCLUDE, "gemv_ops.h")
    if _older((EXTENSION, EXTENSION_STAMP), (os.path.join(CSRC, EXTENSION_SRC), header, os.path.abspath(__file__))):
        return True
    with open(EXTENSION_STAMP) as f:
        return f.read() != _extension_target()


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


def _link_extension(obj: str) -> None:
    tmp = EXTENSION + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, "-L" + LIBDIR, "-lgemv", "-Wl,-rpath,$ORIGIN",
          "-L" + os.path.join(_torch_dir(), "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"],
         "extension link failed")
    os.replace(tmp, EXTENSION)
    with open(EXTENSION_STAMP, "w") as f:
        f.write(_extension_target())


def build(force: bool = False, verbose: bool = False, extra_flags=(), extension: bool = True) -> str:
    """Compile (if needed) and return the path of ``libgemv.so``; with
    ``extension`` (the operators' torch entry points) the module next to it too.
    The library is in place before the extension's errors are raised."""
    with _lock:
        library = force or _stale_library()
        extension = extension and (force or _stale_extension())
        if not library and not extension:
            return LIB
        os.makedirs(OBJDIR, exist_ok=True)
        os.makedirs(LIBDIR, exist_ok=True)
        with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
            extension_obj = ex.submit(_compile_extension) if extension else None
            if library:
                _build_library(ex, verbose, extra_flags)
            if extension:
                _link_extension(extension_obj.result())
        return LIB


def _build_library(ex: ThreadPoolExecutor, verbose: bool, extra_flags) -> None:
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

    objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    _run([exe, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-cudart", "static", "-o", tmp, *objs], "link failed")
    os.replace(tmp, LIB)
    # the native measurement tool, linked against the library just built
    tmp = HOST_TOOL + f".tmp{os.getpid()}"
    _run([exe, *NVCC_FLAGS, *extra_flags, os.path.join(CSRC, HOST_TOOL_SRC), "-o", tmp, "-L" + LIBDIR, "-lgemv",
          "-Xlinker", "-rpath,$ORIGIN"], "measurement tool build failed")
    os.replace(tmp, HOST_TOOL)


def ensure_built() -> str:
    return build(force=False)


def lib_path() -> str:
    return LIB


if __name__ == "__main__":
    print(build(extension=False))
