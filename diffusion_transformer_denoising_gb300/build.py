"""Build libdit.so in-tree with nvcc for sm_103a (one gencode, translation
units compiled in parallel, static CUDA runtime so the library loads on a
machine without a driver for the host-only entry points)."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libdit.so")
# debug variant: device-side bounds checks (-DDIT_DEBUG_BOUNDS) that record a
# failing index in the model's error word instead of touching memory
BUILD_DEBUG = os.path.join(PKG, "_build_debug")
LIB_DEBUG = os.path.join(PKG, "libdit_debug.so")
SOURCES = ["dit_api.cu", "elementwise.cu", "simt_f32.cu", "gemm_tc.cu", "attn_tc.cu", "operators_api.cu", "rope.cu",
           "group_norm.cu", "ffn_api.cu", "rms_norm.cu", "rms_norm_f32.cu", "rms_norm_bf16.cu",
           "rms_norm_f16.cu", "gated_ffn.cu", "grad_norm.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(PKG, "..", "include")]


def _nvcc() -> str:
    n = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(n):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libdit.so")
    return n


def _compile(src: str, extra, build_dir: str = BUILD) -> str:
    obj = os.path.join(build_dir, os.path.splitext(src)[0] + ".o")
    cmd = [_nvcc(), *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def build(verbose: bool = False, extra=(), debug: bool = False) -> str:
    """Compile every CUDA source and link libdit.so (libdit_debug.so with the
    device-side bounds checks when debug); returns its path."""
    build_dir, lib = (BUILD_DEBUG, LIB_DEBUG) if debug else (BUILD, LIB)
    flags = list(extra) + (["-DDIT_DEBUG_BOUNDS"] if debug else [])
    os.makedirs(build_dir, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, flags, build_dir), SOURCES))
    tmp = lib + ".tmp"
    cmd = [_nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    if verbose:
        print(f"built {lib}")
    return lib


if __name__ == "__main__":
    import sys
    build(verbose=True, debug="--debug" in sys.argv)
