"""In-tree build of libbitdelta.so (sm_103a) with nvcc, and of the Python binding
of the decoder-block operators (_binding.so) with g++ on torch's headers.

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


def _inputs_mtime() -> float:
    paths = [os.path.join(CSRC, f) for f in SOURCES + HEADERS + [BINDING_SOURCE]]
    paths.append(os.path.join(INCLUDE, "bitdelta.h"))
    paths.append(os.path.join(INCLUDE, "bitdelta_cache.h"))
    paths.append(os.path.join(INCLUDE, "bitdelta_kmerge.h"))
    paths.append(os.path.join(INCLUDE, "bitdelta_block.h"))
    paths.append(os.path.abspath(__file__))
    return max(os.path.getmtime(p) for p in paths)


def _build_binding() -> None:
    import torch
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
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING_PATH)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    newest = _inputs_mtime()
    if not force and all(os.path.exists(p) and os.path.getmtime(p) >= newest
                         for p in (LIB_PATH, BINDING_PATH)):
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

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_build_binding)
        objs = list(ex.map(compile_one, SOURCES))
        binding.result()
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose_ptxas="-v" in sys.argv))
