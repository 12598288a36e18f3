"""Build the COBS CUDA library (``lib/libcobs.so``) for sm_100a with nvcc, and the native binding of its
paged-cache calls (``lib/_paged-<PyTorch>-<Python>.so``) with the host compiler.

Usage: ``python -m block_sparse_long_summary_b200.build [--force]``.
The library is built in place (objects under ``_build/``) so that it travels with the
source tree; it links the CUDA runtime statically and nothing from PyTorch. The binding links the
library and PyTorch; its name holds the versions it is built for, so that others get their own.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB_DIR = os.path.join(HERE, "lib")
LIB = os.path.join(LIB_DIR, "libcobs.so")
BINDING_SRC = "paged_binding.cpp"
SOURCES = ["api.cu", "summary.cu", "select.cu", "decode.cu", "decode_stream.cu", "decode_step.cu", "tma.cu", "prefill.cu",
           "mass.cu", "basis.cu", "paged_tables.cu", "paged_attn.cu", "paged_simt.cu",
           "paged_chunk.cu", "paged_decode.cu", "paged_decode_f32.cu"]
HEADERS = ["common.cuh", "attn.cuh", "dims.h", "tma.h", "tc.cuh", "select_core.cuh", "stream_tile.cuh",
           "paged.h", "paged_kernels.h", "paged_plan.cuh"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def binding_path() -> str:
    """The binding for the running Python and its PyTorch."""
    import torch
    return os.path.join(LIB_DIR, f"_paged-{torch.__version__}-{sys.implementation.cache_tag}.so")


def _fresh(target: str, sources: list[str]) -> bool:
    files = [os.path.join(CSRC, s) for s in sources if os.path.exists(os.path.join(CSRC, s))]
    files += [os.path.join(ROOT, "include", "cobs.h"), os.path.abspath(__file__)]
    return os.path.exists(target) and os.path.getmtime(target) >= max(os.path.getmtime(f) for f in files)


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, src.replace(".cu", ".o"))
    cmd = [nvcc(), *ARCH, *FLAGS, "-I", os.path.join(ROOT, "include"), "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stderr or r.stdout):
        sys.stderr.write(r.stdout + r.stderr)
    return obj


def _build_binding() -> None:
    """The binding of the paged calls: it finds the library beside itself and PyTorch's libraries in the
    process that imports it."""
    import sysconfig

    from torch.utils import cpp_extension as ext
    tmp = binding_path() + f".tmp{os.getpid()}"
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-w", os.path.join(CSRC, BINDING_SRC), "-o", tmp,
           "-I", sysconfig.get_paths()["include"], "-I", cuda, *[a for d in ext.include_paths() for a in ("-isystem", d)],
           "-L", LIB_DIR, "-lcobs", "-Wl,-rpath,$ORIGIN", *[a for d in ext.library_paths() for a in ("-L", d)],
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    import torch
    cmd.append(f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"building the paged binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, binding_path())


def build(force: bool = False, verbose: bool = False) -> str:
    if force or not _fresh(LIB, SOURCES + HEADERS):
        _build_library(verbose)
    if force or not _fresh(binding_path(), [BINDING_SRC]):
        _build_binding()
    return LIB


def _build_library(verbose: bool) -> None:
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    srcs = [s for s in SOURCES if os.path.exists(os.path.join(CSRC, s))]
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
