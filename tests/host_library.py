"""Builds the library's host sources with host_runtime.cpp, a runtime without a
GPU, and loads them next to the real library."""

from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "sparse_dense_gemm_amd", "csrc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")

X, PARTIALS, COUNTERS, X_ROWS, LAID_OUT, PICKED, ALLOCATIONS = range(7)


def build(folder) -> str:
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir(os.path.join(ROCM, "include", "hip")):
        pytest.skip("needs g++ and the HIP headers")
    out = os.path.join(str(folder), "libspense_host.so")
    src = [os.path.join(CSRC, "spense_api.cpp"), os.path.join(CSRC, "spense_mx_api.cpp"),
           os.path.join(HERE, "host_runtime.cpp")]
    # -Bsymbolic: a HIP runtime that torch has loaded does not take the place of this one
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-w", "-fPIC", "-shared", "-Wl,-Bsymbolic", "-D__HIP_PLATFORM_AMD__",
                        f"-I{ROCM}/include", *src, "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return out


def load(folder) -> ctypes.CDLL:
    lib = ctypes.CDLL(build(folder))
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.host_seen.restype = i64
    lib.host_live.argtypes = [i64]
    lib.host_live_bytes.restype = i64
    lib.spense_pack.argtypes = [vp, i32, i64, i64, i64, vp, vp, i64, ctypes.c_double, vp, ctypes.POINTER(vp)]
    lib.spense_linear.argtypes = [vp, vp, i32, i64, i64, vp, i32, i64, vp]
    lib.spense_linear_w8a8.argtypes = [vp, vp, i64, i64, vp, i32, i64, i32, vp]
    lib.spense_pack_mx4.argtypes = [vp, i64, vp, i64, i64, i64, vp, ctypes.POINTER(vp)]
    lib.spense_linear_w4a4.argtypes = [vp, vp, i64, i64, vp, i32, i64, vp]
    lib.spense_pack_experts.argtypes = [vp, i32, vp, i64, i64, i64, i64, i64, i32, vp, ctypes.POINTER(vp)]
    lib.spense_experts_linear.argtypes = [vp, vp, i32, i64, i64, vp, vp, i64, vp, i32, i64, vp]
    lib.spense_free.argtypes = [vp]
    return lib
