"""Build librtq.so (the HIP kernels + C ABI) in-tree with hipcc for gfx950, and _native.so (the binding of its short calls
to torch tensors) with the host compiler."""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "librtq.so")
NATIVE = os.path.join(PKG, "_native.so")
SOURCES = ["rpbh_rows.hip", "rpbh_quant.hip", "gemm_i8.hip", "gemm_lut.hip", "fp8_rows.hip", "fp8_gemm.hip", "fp8_gemm_large.hip", "fp8_small.hip",
           "fp8_wgrad.hip", "fp8_wgrad_large.hip", "rmsnorm.hip", "glu.hip", "fp8_glu_large.hip", "fp8_glu_tile.hip", "fp8_glu_small.hip", "grads.hip", "rtq_api.cpp", "fp8_api.cpp",
           "block_api.cpp", "rtq_host.cpp", "launch_cache.cpp"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
# Packed fp32 instructions stay off: the compiler must not form v_pk_{add,mul,fma}_f32.
FLAGS = ["-O3", "-std=c++17", "--offload-arch=gfx950", "-fPIC", "-Wall", "-Wno-unused-function",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-fno-gpu-rdc", "-I" + os.path.join(ROOT, "include")]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _build_native() -> str:
    import torch
    base = os.path.dirname(torch.__file__)
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    include = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(rocm, "include")]
    tmp = NATIVE + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *("-isystem" + i for i in include),
           os.path.join(CSRC, "bind.cpp"), "-o", tmp, "-L" + os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-lc10_hip", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"host compiler failed for bind.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, NATIVE)
    return NATIVE


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=8) as ex:
        native = ex.submit(_build_native)
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    native.result()   # raises where the binding failed; the C ABI does not need it
    if verbose:
        print("built", LIB, "and", NATIVE)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
