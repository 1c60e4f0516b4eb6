"""Build libtilegemm.so in-tree with hipcc for gfx950.

    python -m tile_level_gemm_amd.build

Objects go to tile_level_gemm_amd/_build/ (git-ignored); the library lands next to
this file so that it travels with the source tree, and so does the module of the tensor calls
(_tensor_calls.so, host code against torch's headers, linked to the library beside it).
"""

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libtilegemm.so")
CALLS = os.path.join(HERE, "_tensor_calls.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

SOURCES = ["abi.cpp", "plan.cpp", "copy_kernels.hip", "gemm_kernels.hip", "gemm_direct.hip",
           "gemm_direct_kk.hip", "gemm_direct_km.hip", "gemm_direct_mk.hip", "gemm_direct_mm.hip",
           "gemm_fp8.hip", "gemm_fp8_km.hip", "gemm_fp8_mk.hip", "gemm_fp8_mm.hip",
           "gemm_mx_kk.hip", "gemm_mx_km.hip", "gemm_mx_mk.hip", "gemm_mx_mm.hip", "gemm_mx_packed.hip", "gemm_mx_fp4.hip", "gemm_mx_fp6.hip",
           "frag.cpp", "frag_kernels.hip", "async_copy.hip",
           "layer_abi.cpp", "ep_gemm_kk.hip", "ep_gemm_km.hip", "ep_gemm_mk.hip", "ep_gemm_mm.hip",
           "ep_gemm_fp8.hip", "ep_tokens.hip", "ep_kernels.hip", "norm.hip"]

# -packed-fp32-ops: no v_pk_*_f32 in generated code (the device pass honours it; the
# host pass warns that it does not know the feature).
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-mcode-object-version=5",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wall", "-Wno-unused-function", "-I", os.path.join(HERE, "..", "include")]


def _compile(src):
    path = os.path.join(CSRC, src)
    obj = os.path.join(BUILD, src + ".o")
    lang = ["-x", "hip"] if src.endswith(".hip") else []
    cmd = [HIPCC] + FLAGS + lang + ["-c", path, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    err = "\n".join(l for l in r.stderr.splitlines() if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{err}")
    if err.strip():
        sys.stderr.write(err + "\n")
    return obj


def _run(what, cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stderr}")


def _compile_calls():
    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    obj = os.path.join(BUILD, "tensor_calls.cpp.o")
    _run("g++ on tensor_calls.cpp",
         ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          "-I", os.path.join(HERE, "..", "include"), "-isystem", sysconfig.get_paths()["include"],
          "-isystem", os.path.join(root, "include"), "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
          "-isystem", "/opt/rocm/include", "-c", os.path.join(CSRC, "tensor_calls.cpp"), "-o", obj])
    return obj, os.path.join(root, "lib")


def build(jobs=8):
    """Compile every source, link libtilegemm.so and _tensor_calls.so; returns the library path."""
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=jobs) as ex:
        calls = ex.submit(_compile_calls)
        objs = list(ex.map(_compile, SOURCES))
        obj, torch_lib = calls.result()
    tmp = LIB + ".tmp"
    _run("link", [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-Wl,-soname,libtilegemm.so", "-o", tmp] + objs)
    os.replace(tmp, LIB)
    tmp = CALLS + ".tmp"
    # torch is imported before the module, so its own rpath finds torch's libraries
    _run("link of _tensor_calls", ["g++", "-shared", "-o", tmp, obj, "-L", HERE, "-l:libtilegemm.so", "-L", torch_lib,
                                   "-ltorch_python", "-ltorch_hip", "-ltorch_cpu", "-lc10_hip", "-lc10",
                                   "-Wl,-rpath,$ORIGIN"])
    os.replace(tmp, CALLS)
    return LIB


if __name__ == "__main__":
    print(build())
