"""Compile libbsq (the CUDA kernels + C ABI) in-tree for sm_103a with nvcc, and
the compiled part of its Python binding with the host compiler.  The library
needs nothing but the CUDA toolkit (``python fp8_activation_quantization_bsq_gb300/_build.py``);
the binding is built where torch is installed."""
from __future__ import annotations

import importlib.util
import os
import re
import shutil
import subprocess
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
REPO_DIR = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(REPO_DIR, "include")
LIB_DIR = os.path.join(PKG_DIR, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libbsq.so")

SOURCES = ["bsq.cu", "kv_cache.cu", "moe.cu", "linear.cu", "rope.cu", "route.cu"]
HEADERS = ["host_common.h", "host_regions.h", "tcgen05.cuh", "serving_common.cuh", "kv_append.cuh", "kv_attention.cuh", "kv_prompt.cuh", "moe_layer.cuh",
           "packed_linear.cuh", "packed_many.cuh", "qk_norm_rope.cuh", "moe_route.cuh",
           "device_common.cuh", "box_quant.cuh", "dense_quant.cuh", "grouped_quant.cuh", "interleave.cuh",
           "tensor_scale.cuh", "block_scaled_dot.cuh", "cluster.cuh", "gemm_quant.cuh", "grouped_token.cuh"]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libbsq")


def _torch_dir():
    """Where torch is installed (not imported for that), or None."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _binding_path():
    """The binding's file, named by the torch and the Python that it is compiled against, whose classes it holds by layout; None without torch."""
    base = _torch_dir()
    if base is None:
        return None
    with open(os.path.join(base, "version.py")) as f:
        version = re.search(r"^__version__ = ['\"]([^'\"]+)", f.read(), re.M).group(1)
    return os.path.join(LIB_DIR, f"_bsq_binding-{version}{sysconfig.get_config_var('EXT_SUFFIX')}")


BINDING = "binding.cpp"
BINDING_PATH = _binding_path()


def _inputs():
    return ([os.path.join(CSRC, s) for s in SOURCES + HEADERS + [BINDING]]
            + [os.path.join(INCLUDE, "bsq.h"), os.path.abspath(__file__)])


def is_stale() -> bool:
    outputs = [LIB_PATH] + ([BINDING_PATH] if BINDING_PATH else [])
    if not all(os.path.exists(p) for p in outputs):
        return True
    t = min(os.path.getmtime(p) for p in outputs)
    return any(os.path.getmtime(p) > t for p in _inputs())


def _binding_commands():
    """Compile and link commands of the binding: torch's headers and libraries, libbsq beside it."""
    base = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    obj = os.path.join(LIB_DIR, BINDING + ".o")
    cxx = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE, "-isystem", os.path.join(base, "include"), "-isystem",
           os.path.join(base, "include", "torch", "csrc", "api", "include"), "-isystem", os.path.join(cuda, "include"), "-isystem",
           sysconfig.get_paths()["include"], "-c", "-o", obj, os.path.join(CSRC, BINDING)]
    link = ["g++", "-shared", "-o", BINDING_PATH + ".tmp", obj, "-L" + LIB_DIR, "-lbsq", "-L" + os.path.join(base, "lib"), "-ltorch_python",
            "-ltorch_cpu", "-ltorch", "-ltorch_cuda", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    return cxx, link


def build(force: bool = False, verbose: bool = False) -> str:
    """Build ``_lib/libbsq.so`` and, with torch, the binding beside it (skipped when up to date); returns the library's path."""
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
    if BINDING_PATH:
        binding, binding_link = _binding_commands()
        jobs.append(binding)
    running = [subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True) for c in jobs]
    results = [(c, p.communicate()[0], p.returncode) for c, p in zip(jobs, running)]
    def then(command):
        res = subprocess.run(command, capture_output=True, text=True)
        results.append((command, res.stdout + res.stderr, res.returncode))

    if all(rc == 0 for _, _, rc in results):
        then(base + ["-shared", "-Xlinker", "-rpath,/usr/local/cuda/lib64", "-Xlinker", "-soname,libbsq.so", "-o", tmp] + objects)
    if all(rc == 0 for _, _, rc in results):
        os.replace(tmp, LIB_PATH)
        if BINDING_PATH:
            then(binding_link)
    for cmd, text, rc in results:
        if verbose or rc != 0:
            print(" ".join(cmd))
            print(text)
    failed = [text for _, text, rc in results if rc != 0]
    if failed:
        raise RuntimeError("libbsq build failed:\n" + "\n".join(failed)[-4000:])
    if BINDING_PATH:
        os.replace(BINDING_PATH + ".tmp", BINDING_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
