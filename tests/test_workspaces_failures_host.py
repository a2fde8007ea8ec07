"""Workspaces of a handle after a call that could not grow them, looked at on the
host: the library's host code with a runtime that hands out addresses and fails
when it is told to."""

import ctypes
import os
import shutil
import subprocess

import pytest

import host_library as hl
import sparse_dense_gemm_amd as sdg

P = 1 << 20      # a 16-byte aligned address that nothing dereferences
STREAM = 1 << 12
N, K = 64, 8192  # few row tiles, many columns: small calls split K
F32, BF16, FP8 = sdg.DT_F32, sdg.DT_BF16, sdg.DT_FP8
ZERO = "_ZN6spense15launch_zero_i32EPilP12ihipStream_t"


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir(os.path.join(hl.ROCM, "include", "hip")):
        pytest.skip("needs g++ and the HIP headers")
    out = os.path.join(str(tmp_path_factory.mktemp("failing")), "libspense_failing.so")
    src = [os.path.join(hl.CSRC, f) for f in ("spense_api.cpp", "spense_mx_api.cpp", "spense_fp8b_api.cpp")]
    src += [os.path.join(hl.HERE, f) for f in ("host_runtime.cpp", "fp8b_host_runtime.cpp", "failing_runtime.cpp")]
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-w", "-fPIC", "-shared", "-Wl,-Bsymbolic", "-Wl,--wrap=hipMalloc", "-Wl,--wrap=hipGetLastError",
                        f"-Wl,--wrap={ZERO}", "-D__HIP_PLATFORM_AMD__", f"-I{hl.ROCM}/include", *src, "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    lib = ctypes.CDLL(out)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    for f in ("host_seen8", "host_seen", "host_live_bytes", "host_zeroed"):
        getattr(lib, f).restype = i64
    lib.host_fail_alloc.argtypes = [i64]
    lib.spense_pack.argtypes = [vp, i32, i64, i64, i64, vp, vp, i64, ctypes.c_double, vp, ctypes.POINTER(vp)]
    lib.spense_pack_mx4.argtypes = [vp, i64, vp, i64, i64, i64, vp, ctypes.POINTER(vp)]
    lib.spense_pack_experts.argtypes = [vp, i32, vp, i64, i64, i64, i64, i64, i32, vp, ctypes.POINTER(vp)]
    lib.spense_pack_fp8b.argtypes = [vp, i64, vp, i64, i64, i64, vp, ctypes.POINTER(vp)]
    lib.spense_pack_experts_fp8b.argtypes = [vp, vp, i64, i64, i64, i64, i64, i32, vp, ctypes.POINTER(vp)]
    lib.spense_linear.argtypes = [vp, vp, i32, i64, i64, vp, i32, i64, vp]
    lib.spense_linear_w8a8.argtypes = [vp, vp, i64, i64, vp, i32, i64, i32, vp]
    lib.spense_linear_w4a4.argtypes = [vp, vp, i64, i64, vp, i32, i64, vp]
    lib.spense_experts_linear.argtypes = [vp, vp, i32, i64, i64, vp, vp, i64, vp, i32, i64, vp]
    lib.spense_free.argtypes = [vp]
    return lib


def sparse(lib, h):
    return lib.spense_pack(P, FP8, N, K, K, P, None, 0, 0.25, None, ctypes.byref(h))


def mx4(lib, h):
    return lib.spense_pack_mx4(P, K // 2, P, K // 32, N, K, None, ctypes.byref(h))


def experts(lib, h):
    return lib.spense_pack_experts(P, BF16, None, 4, N, K, K, 0, 0, None, ctypes.byref(h))


def fp8b(lib, h):
    return lib.spense_pack_fp8b(P, K, P, K // 128, N, K, None, ctypes.byref(h))


def fp8b_experts(lib, h):
    return lib.spense_pack_experts_fp8b(P, P, 4, N, K, K, K // 128, 0, None, ctypes.byref(h))


def linear(lib, h, M):
    return lib.spense_linear(h, P, BF16, M, K, P, F32, N, STREAM)


def grouped(adtype):
    return lambda lib, h, M: lib.spense_experts_linear(h, P, adtype, M, K, None, P, M, P, F32, N, STREAM)


CALLS = {
    "sparse": (sparse, linear),
    "sparse w8a8": (sparse, lambda lib, h, M: lib.spense_linear_w8a8(h, P, M, K, P, F32, N, 0, STREAM)),
    "mx4": (mx4, linear),
    "mx4 w4a4": (mx4, lambda lib, h, M: lib.spense_linear_w4a4(h, P, M, K, P, F32, N, STREAM)),
    "experts": (experts, grouped(BF16)),
    "fp8b": (fp8b, linear),
    "fp8b w8a8": (fp8b, lambda lib, h, M: lib.spense_linear_w8a8(h, P, M, K, P, F32, N, 0, STREAM)),
    "fp8b experts": (fp8b_experts, grouped(BF16)),
    "fp8b experts call": (fp8b_experts, grouped(FP8)),
}


def pack(lib, make):
    h = ctypes.c_void_p()
    assert make(lib, h) == 0
    return h


def counters(lib):
    return lib.host_seen8(3) or lib.host_seen(hl.COUNTERS)


@pytest.mark.parametrize("kind", CALLS)
def test_counters_are_zeroed_before_they_are_used(lib, kind):
    """A call whose zeroing failed leaves no counters that a later one takes as they are."""
    make, run = CALLS[kind]
    h = pack(lib, make)
    lib.host_fail_zero(2)
    for _ in range(2):
        assert run(lib, h, 4) != 0
    lib.host_forget()
    lib.host_forget8()
    assert run(lib, h, 4) == 0
    assert counters(lib) and counters(lib) == lib.host_zeroed()
    lib.spense_free(h)
    assert lib.host_live_bytes() == 0


@pytest.mark.parametrize("kind", CALLS)
@pytest.mark.parametrize("bytes_", [1, 1 << 12, 1 << 16], ids=["any", "4K", "64K"])
def test_a_failed_call_takes_nothing_from_the_others(lib, kind, bytes_):
    """What could be captured before a call that could not grow the workspaces still can after it."""
    make, run = CALLS[kind]

    def capturable(sizes):
        lib.host_capturing(1)
        good = [M for M in sizes if run(lib, h, M) == 0]
        lib.host_capturing(0)
        return good

    for first, larger in ((64, 700), (700, 5000), (3000, 8000), (9000, 20000)):
        h = pack(lib, make)
        assert run(lib, h, first) == 0
        sizes = range(1, first + 1, 1 + first // 200)
        before = capturable(sizes)
        assert before
        held = lib.host_live_bytes()
        lib.host_fail_alloc(bytes_)
        failed = run(lib, h, larger) != 0  # where it needs an allocation of that size
        lib.host_fail_alloc(0)
        assert capturable(sizes) == before, (kind, first, larger)
        assert not failed or lib.host_live_bytes() >= held
        lib.spense_free(h)
    assert lib.host_live_bytes() == 0


@pytest.mark.parametrize("kind", CALLS)
def test_errors_are_taken_from_the_runtime(lib, kind):
    """A failure is reported once: no later launch of the thread finds it."""
    make, run = CALLS[kind]
    h = ctypes.c_void_p()
    lib.host_fail_alloc(1)
    assert make(lib, h) == sdg.SPENSE_ENOMEM and not h.value
    assert lib.host_last_error() == 0
    h = pack(lib, make)
    lib.host_fail_alloc(1)
    assert run(lib, h, 4) == sdg.SPENSE_ENOMEM
    assert lib.host_last_error() == 0
    lib.host_fail_zero(1)
    assert run(lib, h, 4) == sdg.SPENSE_EHIP
    assert lib.host_last_error() == 0 and lib.spense_last_hip_error() != 0
    assert run(lib, h, 4) == 0
    lib.spense_free(h)
    assert lib.host_live_bytes() == 0
