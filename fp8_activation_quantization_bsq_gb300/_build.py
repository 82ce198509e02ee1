"""Compile libbsq (the CUDA kernels + C ABI) in-tree for sm_103a with nvcc."""
from __future__ import annotations

import os
import shutil
import subprocess

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
REPO_DIR = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(REPO_DIR, "include")
LIB_DIR = os.path.join(PKG_DIR, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libbsq.so")

SOURCES = ["bsq.cu", "kv_cache.cu", "moe.cu", "linear.cu", "rope.cu", "route.cu"]
HEADERS = ["host_common.h", "tcgen05.cuh", "serving_common.cuh", "kv_append.cuh", "kv_attention.cuh", "kv_prompt.cuh", "moe_layer.cuh",
           "packed_linear.cuh", "packed_many.cuh", "qk_norm_rope.cuh", "moe_route.cuh",
           "device_common.cuh", "box_quant.cuh", "dense_quant.cuh", "grouped_quant.cuh", "interleave.cuh",
           "tensor_scale.cuh", "block_scaled_dot.cuh", "cluster.cuh", "gemm_quant.cuh", "grouped_token.cuh"]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libbsq")


def _inputs():
    return ([os.path.join(CSRC, s) for s in SOURCES + HEADERS]
            + [os.path.join(INCLUDE, "bsq.h"), os.path.abspath(__file__)])


def is_stale() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    return any(os.path.getmtime(p) > t for p in _inputs())


def build(force: bool = False, verbose: bool = False) -> str:
    """Build ``_lib/libbsq.so`` (skipped when up to date); returns its path."""
    if not force and not is_stale():
        return LIB_PATH
    os.makedirs(LIB_DIR, exist_ok=True)
    tmp = LIB_PATH + ".tmp"
    base = [nvcc_path(), "-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo",
            "-std=c++17", "-Werror", "all-warnings", "-cudart", "shared", "-Xcompiler", "-fPIC,-fvisibility=hidden",
            "-I", INCLUDE]
    # one compiler process per translation unit, all at once, then the link
    objects = [os.path.join(LIB_DIR, s + ".o") for s in SOURCES]
    jobs = [base + ["-c", "-o", o, os.path.join(CSRC, s)] for s, o in zip(SOURCES, objects)]
    running = [subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True) for c in jobs]
    results = [(c, p.communicate()[0], p.returncode) for c, p in zip(jobs, running)]
    if all(rc == 0 for _, _, rc in results):
        link = base + ["-shared", "-Xlinker", "-rpath,/usr/local/cuda/lib64", "-o", tmp] + objects
        res = subprocess.run(link, capture_output=True, text=True)
        results.append((link, res.stdout + res.stderr, res.returncode))
    for cmd, text, rc in results:
        if verbose or rc != 0:
            print(" ".join(cmd))
            print(text)
    failed = [text for _, text, rc in results if rc != 0]
    if failed:
        raise RuntimeError("libbsq build failed:\n" + "\n".join(failed)[-4000:])
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
