"""Build libfconv.so in-tree with nvcc for sm_103a (GB300).

Each translation unit compiles in parallel into `_build/`, then nvcc links the shared
library next to this file. No CMake, no PyTorch extension machinery: the library has a
plain C ABI (include/fconv.h).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libfconv.so")

SOURCES = ["fconv_api.cpp", "k_direct.cu", "k_depthwise.cu", "k_grouped.cu", "k_igemm_tc.cu",
           "k_igemm_patch.cu", "k_igemm_tf32.cu", "k_transposed.cu", "fconv_noalloc.cu",
           "ops/ops_api.cpp", "ops/k_norm.cu", "ops/k_rope.cu", "ops/k_attn_mma.cu",
           "ops/k_attn_mma_wide.cu", "ops/k_attn_tc_fwd.cu", "ops/k_attn_tc_bwd.cu",
           "ops/block_api.cpp", "ops/k_norm_rope.cu", "ops/k_mlp_mma.cu", "ops/k_mlp_sums.cu",
           "ops/k_mlp_tc.cu", "ops/k_mlp_few.cu",
           "ops/k_mlp_prep.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    path = shutil.which("nvcc")
    if path:
        return path
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: the FusedConv CUDA library cannot be built")


def _deps_mtime() -> float:
    t = 0.0
    for d in (CSRC, os.path.join(CSRC, "ops"), os.path.join(ROOT, "include")):
        for f in os.listdir(d):
            t = max(t, os.path.getmtime(os.path.join(d, f)))
    return t


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0].replace("/", "_") + ".o")
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
           "-I", os.path.join(ROOT, "include"), *extra, "-c", os.path.join(CSRC, src),
           "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile (if sources changed) and return the path of libfconv.so."""
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _deps_mtime():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra), SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True))
