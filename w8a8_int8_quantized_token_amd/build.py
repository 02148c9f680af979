"""Build libw8a8.so (HIP, gfx950) and _calls.so (the binding's native calls,
host code against torch's headers) in-tree with hipcc and g++.

Usage: python w8a8_int8_quantized_token_amd/build.py
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libw8a8.so")
CALLS = os.path.join(PKG, "_calls.so")
SOURCES = ["quantize_rows.hip", "dequantize_rows.hip", "gemm_i8.hip", "splitk_reduce.hip",
           "mfma_ceiling.hip", "w8a8_api.hip", "gemm_gated.hip", "gemm_gated_grad.hip", "gemm_bf16.hip",
           "backward_layout.hip", "few_grad.hip", "few_tokens.hip", "qk_norm_rope.hip", "block_api.hip"]
ARCH = "gfx950"

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    # every fp32 operation is rounded on its own unless written as an fma
    "-ffp-contract=off",
    # no packed fp32 instructions in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-command-line-argument",
    "-I", os.path.join(ROOT, "include"),
]


def _compile(src: str) -> str:
    obj = os.path.join(OBJ, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


def _run(cmd: list[str], what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stderr}")


def _calls_object() -> str:
    """The native calls, compiled (they need only torch's headers)."""
    import torch
    from torch.utils import cpp_extension

    obj = os.path.join(OBJ, "torch_calls.o")
    rocm = os.path.dirname(os.path.dirname(HIPCC))
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          *[f"-I{p}" for p in cpp_extension.include_paths()], f"-I{sysconfig.get_paths()['include']}",
          f"-I{rocm}/include", "-c", os.path.join(CSRC, "torch_calls.cpp"), "-o", obj], "g++ for torch_calls.cpp")
    return obj


def _link_calls(obj: str) -> None:
    from torch.utils import cpp_extension

    libs = [p for p in cpp_extension.library_paths() if os.path.basename(p) == "lib"]
    tmp = CALLS + ".tmp%d" % os.getpid()
    _run(["g++", "-shared", "-o", tmp, obj, *[f"-L{p}" for p in libs], f"-L{PKG}", "-lc10", "-lc10_hip", "-ltorch_cpu",
          "-ltorch_hip", "-ltorch_python", "-l:libw8a8.so", "-Wl,-rpath,$ORIGIN"], "link of _calls.so")
    os.replace(tmp, CALLS)


def build(verbose: bool = False) -> str:
    os.makedirs(OBJ, exist_ok=True)
    with cf.ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        calls = ex.submit(_calls_object)
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp%d" % os.getpid()
    # (the soname is what _calls.so looks for beside itself)
    _run([HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-Wl,-soname,libw8a8.so", "-o", tmp, *objs], "link")
    os.replace(tmp, LIB)
    _link_calls(calls.result())
    if verbose:
        print(LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
