"""The launches of the fp8b products, looked at on the host: a launch is the one
that its plan priced, for every number of rows that shares the plan."""

import ctypes
import os
import shutil
import subprocess

import pytest

import host_library as hl
import sparse_dense_gemm_amd as sdg

P = 1 << 20  # a 16-byte aligned address that nothing dereferences
STREAM, CONFIG, SPLITS, LAUNCHES = range(4)
LAUNCH = "_ZN6spense18launch_fp8b_linearERKNS_8Fp8bDescERKNS_8Fp8bArgsERKNS_11ExpertsPlanEP12ihipStream_t"
BF16, FP8 = sdg.DT_BF16, sdg.DT_FP8


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir(os.path.join(hl.ROCM, "include", "hip")):
        pytest.skip("needs g++ and the HIP headers")
    out = os.path.join(str(tmp_path_factory.mktemp("launches")), "libspense_launches.so")
    src = [os.path.join(hl.CSRC, f) for f in ("spense_api.cpp", "spense_mx_api.cpp", "spense_fp8b_api.cpp")]
    src += [os.path.join(hl.HERE, f) for f in ("host_runtime.cpp", "fp8b_host_runtime.cpp", "launch_runtime.cpp")]
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-w", "-fPIC", "-shared", "-Wl,-Bsymbolic", f"-Wl,--wrap={LAUNCH}",
                        "-D__HIP_PLATFORM_AMD__", f"-I{hl.ROCM}/include", *src, "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    lib = ctypes.CDLL(out)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.host_told.restype = i64
    lib.spense_pack_fp8b.argtypes = [vp, i64, vp, i64, i64, i64, vp, ctypes.POINTER(vp)]
    lib.spense_pack_experts_fp8b.argtypes = [vp, vp, i64, i64, i64, i64, i64, i32, vp, ctypes.POINTER(vp)]
    lib.spense_linear.argtypes = [vp, vp, i32, i64, i64, vp, i32, i64, vp]
    lib.spense_experts_linear.argtypes = [vp, vp, i32, i64, i64, vp, vp, i64, vp, i32, i64, vp]
    lib.spense_free.argtypes = [vp]
    return lib


def told(lib, call):
    n = lib.host_told(LAUNCHES)
    assert call() == 0 and lib.host_told(LAUNCHES) == n + 1
    return tuple(lib.host_told(f) for f in (STREAM, CONFIG, SPLITS))


@pytest.mark.parametrize("E,N,K", [(16, 3200, 5120), (64, 800, 5120), (8, 3200, 5120), (1, 25600, 5120), (128, 1024, 1024)])
@pytest.mark.parametrize("adtype,yt", [(BF16, BF16), (FP8, BF16), (FP8, sdg.DT_F32)])
def test_rows_of_one_plan_have_one_launch(lib, E, N, K, adtype, yt):
    h = ctypes.c_void_p()
    if E == 1 and adtype == BF16:
        assert lib.spense_pack_fp8b(P, K, P, K // 128, N, K, None, ctypes.byref(h)) == 0
        call = lambda R: lib.spense_linear(h, P, BF16, R, K, P, yt, N, None)
    else:
        assert lib.spense_pack_experts_fp8b(P, P, E, N, K, K, K // 128, 1, None, ctypes.byref(h)) == 0
        call = lambda R: lib.spense_experts_linear(h, P, adtype, R, K, None, P, R, P, yt, N // 2, None)
    seen = {}
    for R in range(1, 1300):
        seen.setdefault((R + 15) // 16, set()).add(told(lib, lambda: call(R)))
    assert all(len(s) == 1 for s in seen.values()), [(16 * r, s) for r, s in seen.items() if len(s) > 1][:4]
    assert any(s for t in seen.values() for s, _, _ in t)  # few rows of such weights are streamed
    for r, launches in seen.items():
        for s, config, _ in launches:
            m_tiles = (1, 2, 4, 8, 8)[config]
            most = 16 * m_tiles if E == 1 else 8 * m_tiles * min(E, 16 * r)
            large = min(E, 16 * r) * N * K > 96 << 20
            assert bool(s) == (m_tiles < 8 and large and 16 * r <= most), (r, s, config)
    lib.spense_free(h)
