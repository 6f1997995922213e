"""Build the CUDA library in-tree: fp8_w8a8_quantized_gb300/_build/libfp8w8a8.so,
and the extension modules of the attention block's and the expert block's
binding beside it.

Each .cu file is compiled for sm_103a only (``-gencode
arch=compute_103a,code=sm_103a``), in parallel, then linked with the static
CUDA runtime into one shared library that exports the C ABI of
include/fp8w8a8.h.  No fast-math: the quantizer's divisions must be IEEE.

Usage: python -m fp8_w8a8_quantized_gb300.build [--verbose]
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.machinery
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB_NAME = "libfp8w8a8.so"
LIB_PATH = os.path.join(OUT_DIR, LIB_NAME)

SOURCES = ["api.cu", "quant.cu", "quant_variants.cu", "norm_quant.cu", "gemm_pair.cu", "gemm_decode.cu", "gemm_blockwise.cu", "noalloc.cu",
           "selftest.cu", "attention_api.cu", "kv_slots.cu", "norm_rope.cu", "attention_prompt.cu", "attention_decode.cu",
           "attention_prefix.cu", "experts_api.cu", "moe_route.cu", "gemm_grouped.cu", "residual_norm.cu"]
HEADERS = ["ptx.cuh", "launch.h", "quant_math.cuh", "decode_common.cuh", "attention_plan.h", "attention_tile.cuh",
           "grouped_plan.h"]

# The binding's extension modules (host code only; they link the library and torch).
MODULES = ["attention_binding", "experts_binding"]
MODULE_HEADERS = ["binding_args.h"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + [
    "-O3", "-std=c++17", "-lineinfo",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-I", INCLUDE, "-I", CSRC,
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(OUT_DIR, src.replace(".cu", ".o"))
    deps = [os.path.join(CSRC, src)] + [os.path.join(CSRC, h) for h in HEADERS] + [
        os.path.join(INCLUDE, "fp8w8a8.h"), __file__]
    if not verbose and not _stale(obj, deps):
        return obj
    cmd = [nvcc()] + NVCC_FLAGS + (["-Xptxas", "-v"] if verbose else []) + [
        "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and r.stderr:
        sys.stderr.write(r.stderr)
    return obj


def _compile_module(name: str) -> str:
    import torch
    src = os.path.join(CSRC, name + ".cpp")
    obj = os.path.join(OUT_DIR, name + ".o")
    deps = [src] + [os.path.join(CSRC, h) for h in MODULE_HEADERS] + [
        os.path.join(INCLUDE, "fp8w8a8.h"), __file__, torch.__file__]
    if not _stale(obj, deps):
        return obj
    troot = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           "-I", INCLUDE, "-I", os.path.join(troot, "include"),
           "-I", os.path.join(troot, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-I", cuda, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {name}.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_module(name: str, obj: str) -> None:
    import torch
    path = os.path.join(OUT_DIR, "fp8_" + name + importlib.machinery.EXTENSION_SUFFIXES[0])
    if not _stale(path, [obj, LIB_PATH]):
        return
    tmp = path + f".{os.getpid()}.tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", OUT_DIR, f"-l:{LIB_NAME}", "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(os.path.dirname(torch.__file__), "lib"),
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding module failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)


def build(verbose: bool = False) -> str:
    """Compile (incrementally) and link the library and the binding's modules;
    returns the library's path."""
    os.makedirs(OUT_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + len(MODULES)) as ex:
        modules = [ex.submit(_compile_module, m) for m in MODULES]
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    if _stale(LIB_PATH, objs):
        tmp = LIB_PATH + f".{os.getpid()}.tmp"
        cmd = [nvcc()] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB_PATH)
    for name, obj in zip(MODULES, modules):
        _link_module(name, obj.result())
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv))
