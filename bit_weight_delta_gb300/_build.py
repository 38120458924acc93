"""In-tree build of libbitdelta.so (sm_103a) with nvcc, and of the Python binding
of the decoder-block operators (_binding.so) with g++ on torch's headers.  The
library needs neither g++ nor torch's headers, and is built without them.

Each .cu file compiles to an object in parallel, then nvcc links the shared
library next to this file.  The CUDA runtime is linked statically; the driver
API is reached at run time through the runtime's entry-point query, so the
library loads on a host without a GPU (for symbol checks) and needs no -lcuda.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build", "bitdelta")
LIB_PATH = os.path.join(HERE, "libbitdelta.so")
BINDING_PATH = os.path.join(HERE, "_binding.so")
BINDING_SOURCE = "binding.cpp"
BINDING_STAMP = os.path.join(BUILD_DIR, "binding.txt")  # what _binding.so was built for

SOURCES = ["abi.cu", "compress.cu", "reconstruct.cu", "gemv.cu", "gemm_pair.cu", "cache.cu",
           "kmerge.cu", "similarity.cu", "monosoup.cu", "add_norm.cu", "kv_append.cu",
           "attention.cu", "attn_decode.cu", "attn_tile.cu"]
HEADERS = ["common.cuh", "kernels.h", "gemm_common.cuh", "split_schedule.h", "attention.cuh", "attn_decode.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
              "-I", CSRC]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _current(out: str, sources, headers) -> bool:
    """Whether `out` is newer than these files and this one."""
    paths = [os.path.join(CSRC, f) for f in sources] + [os.path.join(INCLUDE, f) for f in headers]
    paths.append(os.path.abspath(__file__))
    return os.path.exists(out) and os.path.getmtime(out) >= max(map(os.path.getmtime, paths))


def _binding_for() -> str:
    """What a binary on torch's C++ classes is bound to."""
    import torch
    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"


def _stamp() -> str:
    try:
        with open(BINDING_STAMP) as f:
            return f.read()
    except OSError:
        return ""


def build_binding(force: bool = False) -> str:
    import torch
    if not force and _stamp() == _binding_for() and _current(
            BINDING_PATH, [BINDING_SOURCE], ["bitdelta.h", "bitdelta_block.h"]):
        return BINDING_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    base = os.path.dirname(torch.__file__)
    lib = os.path.join(base, "lib")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", INCLUDE,
           "-I", os.path.join(base, "include"),
           "-I", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-I", os.path.join(cuda, "include"), "-I", sysconfig.get_paths()["include"],
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           os.path.join(CSRC, BINDING_SOURCE), "-o", tmp, "-L", lib, "-lc10", "-ltorch_cpu",
           "-ltorch_python", "-ltorch_cuda", "-lc10_cuda", f"-Wl,-rpath,{lib}"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        raise RuntimeError(f"g++ is needed for {BINDING_SOURCE}: {e}") from e
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING_PATH)
    with open(BINDING_STAMP, "w") as f:
        f.write(_binding_for())
    return BINDING_PATH


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """The C library."""
    if not force and _current(LIB_PATH, SOURCES + HEADERS,
                              ["bitdelta.h", "bitdelta_cache.h", "bitdelta_kmerge.h",
                               "bitdelta_block.h"]):
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose_ptxas:
            print(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def build_all(force: bool = False, verbose_ptxas: bool = False) -> str:
    """The library and the binding, side by side."""
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        binding = ex.submit(build_binding, force)
        path = build(force, verbose_ptxas)
        binding.result()
    return path


if __name__ == "__main__":
    import sys
    print(build_all(force=True, verbose_ptxas="-v" in sys.argv))
