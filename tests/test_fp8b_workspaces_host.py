"""Workspaces of an fp8b handle, looked at on the host: the library's host code
with a runtime that only hands out addresses."""

import ctypes
import os
import shutil
import subprocess

import pytest

import host_library as hl
import sparse_dense_gemm_amd as sdg

P = 1 << 20      # a 16-byte aligned address that nothing dereferences
STREAM = 1 << 12
N, K = 64, 8192  # few row tiles, many columns: small calls split K and need partial sums and counters
BLOCKS = K // 128
X, SCALES, PARTIALS, COUNTERS, X_ROWS, LAID_OUT = range(6)


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir(os.path.join(hl.ROCM, "include", "hip")):
        pytest.skip("needs g++ and the HIP headers")
    out = os.path.join(str(tmp_path_factory.mktemp("host8")), "libspense_host8.so")
    src = [os.path.join(hl.CSRC, f) for f in ("spense_api.cpp", "spense_mx_api.cpp", "spense_fp8b_api.cpp")]
    src += [os.path.join(hl.HERE, f) for f in ("host_runtime.cpp", "fp8b_host_runtime.cpp")]
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-w", "-fPIC", "-shared", "-Wl,-Bsymbolic", "-D__HIP_PLATFORM_AMD__",
                        f"-I{hl.ROCM}/include", *src, "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    lib = ctypes.CDLL(out)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.host_seen8.restype = lib.host_seen.restype = lib.host_live_bytes.restype = i64
    lib.host_live.argtypes = [i64]
    lib.spense_linear.argtypes = [vp, vp, i32, i64, i64, vp, i32, i64, vp]
    lib.spense_linear_w8a8.argtypes = [vp, vp, i64, i64, vp, i32, i64, i32, vp]
    lib.spense_pack_fp8b.argtypes = [vp, i64, vp, i64, i64, i64, vp, ctypes.POINTER(vp)]
    lib.spense_linear_fp8b.argtypes = [vp, vp, i64, vp, i64, i64, vp, i32, i64, vp]
    lib.spense_pack_experts_fp8b.argtypes = [vp, vp, i64, i64, i64, i64, i64, i32, vp, ctypes.POINTER(vp)]
    lib.spense_experts_linear.argtypes = [vp, vp, i32, i64, i64, vp, vp, i64, vp, i32, i64, vp]
    lib.spense_experts_linear_fp8b.argtypes = [vp, vp, i64, vp, i64, i64, vp, vp, i64, vp, i32, i64, vp]
    lib.spense_info.argtypes = [vp, ctypes.POINTER(sdg.LayerInfo)]
    lib.spense_free.argtypes = [vp]
    return lib


def layer(lib):
    h = ctypes.c_void_p()
    assert lib.spense_pack_fp8b(P, K, P, BLOCKS, N, K, None, ctypes.byref(h)) == 0
    return h


def experts(lib, glu=0, n=N):
    h = ctypes.c_void_p()
    assert lib.spense_pack_experts_fp8b(P, P, 4, n, K, K, BLOCKS, glu, None, ctypes.byref(h)) == 0
    return h


F32, BF16, FP8 = sdg.DT_F32, sdg.DT_BF16, sdg.DT_FP8
CALLS = {
    "linear": (layer, lambda lib, h, M, yt=F32, x=P, ld=K: lib.spense_linear(h, x, BF16, M, ld, P, yt, N, STREAM)),
    "w8a8": (layer, lambda lib, h, M, yt=F32, x=P, ld=K: lib.spense_linear_w8a8(h, x, M, ld, P, yt, N, 0, STREAM)),
    "codes": (layer, lambda lib, h, M, yt=F32, x=P, ld=K: lib.spense_linear_fp8b(h, x, ld, P, BLOCKS, M, P, yt, N, STREAM)),
    "experts": (experts, lambda lib, h, M, yt=F32, x=P, ld=K, rows=None, R=None:
                lib.spense_experts_linear(h, x, BF16, M, ld, rows, P, M if R is None else R, P, yt, N, STREAM)),
    "experts call": (experts, lambda lib, h, M, yt=F32, x=P, ld=K, rows=None, R=None:
                     lib.spense_experts_linear(h, x, FP8, M, ld, rows, P, M if R is None else R, P, yt, N, STREAM)),
    "experts codes": (experts, lambda lib, h, M, yt=F32, x=P, ld=K, rows=None, R=None:
                      lib.spense_experts_linear_fp8b(h, x, ld, P, BLOCKS, M, rows, P, M if R is None else R, P, yt, N,
                                                     STREAM)),
}


def pointers(lib, run, h, M, **kw):
    """Workspaces that the launch of a call at M rows was given."""
    lib.host_forget8()
    assert run(lib, h, M, **kw) == 0
    return [p for p in (lib.host_seen8(f) for f in (X, SCALES, PARTIALS, COUNTERS)) if p not in (0, P, P + 1)]


def base(lib, p):
    """Whether p lies in a live allocation (a workspace's scales follow its codes)."""
    return lib.host_live(p) or any(lib.host_live(q) for q in range(p - p % 4096, p - (1 << 27), -4096))


@pytest.mark.parametrize("kind", CALLS)
@pytest.mark.parametrize("x", [P, P + 1], ids=["in place", "laid out"])
def test_captured_workspaces_outlive_larger_calls(lib, kind, x):
    pack, run = CALLS[kind]
    before = lib.host_live_bytes()
    h = pack(lib)
    pointers(lib, run, h, 4, x=x)
    lib.host_capturing(1)
    recorded = pointers(lib, run, h, 4, x=x)
    lib.host_capturing(0)
    assert recorded and all(base(lib, p) for p in recorded)
    moved = set()
    for M in (64, 700, 5000):
        moved |= set(pointers(lib, run, h, M, x=x)) - set(recorded)
        assert all(base(lib, p) for p in recorded), M
    assert moved
    lib.spense_free(h)
    assert lib.host_live_bytes() == before


@pytest.mark.parametrize("kind", CALLS)
def test_smaller_calls_need_no_more(lib, kind):
    """After one eager call every smaller one, with either output type, can be captured."""
    pack, run = CALLS[kind]
    for x in (P, P + 1):
        for first in (F32, BF16):
            h = pack(lib)
            assert run(lib, h, 3000, yt=first, x=x) == 0
            lib.host_capturing(1)
            for yt in (F32, BF16):
                for M in list(range(1, 200)) + list(range(200, 3001, 61)):
                    assert run(lib, h, M, yt=yt, x=x) == 0, (kind, M, yt)
            lib.host_capturing(0)
            lib.spense_free(h)


@pytest.mark.parametrize("kind", ["experts", "experts call", "experts codes"])
def test_only_rows_that_are_read_are_laid_out(lib, kind):
    """Picked rows: the R that are read, or X's own if it has no more."""
    _, run = CALLS[kind]
    for M, R, want in ((5000, 40, 40), (30, 200, 30)):
        h = experts(lib)
        lib.host_forget8()
        lib.host_forget()
        assert run(lib, h, M, x=P + 1, rows=P, R=R) == 0
        laid = lib.host_seen8(LAID_OUT) or lib.host_seen(hl.LAID_OUT)
        assert laid == want and lib.host_seen8(X_ROWS) == want
        lib.spense_free(h)


def test_aligned_activations_are_read_in_place(lib):
    for kind in ("linear", "codes", "experts", "experts codes"):
        pack, run = CALLS[kind]
        h = pack(lib)
        lib.host_forget8()
        assert run(lib, h, 33) == 0 and lib.host_seen8(X) == P, kind
        assert run(lib, h, 33, ld=K + 1) == 0 and lib.host_seen8(X) != P, kind
        # the kernel's offsets reach 256 rows of codes that far apart, but not of bf16
        assert run(lib, h, 33, ld=(1 << 23) - 16) == 0 and (lib.host_seen8(X) == P) == ("codes" in kind), kind
        lib.spense_free(h)


def test_strides_of_scales(lib):
    """Scales far apart are laid out first; a stride whose products could leave 64 bits is refused."""
    for kind in ("codes", "experts codes"):
        h = CALLS[kind][0](lib)
        for lds, want in (((1 << 21) - 1, True), (1 << 21, False), ((1 << 23) - 1, False)):
            lib.host_forget8()
            if kind == "codes":
                assert lib.spense_linear_fp8b(h, P, K, P, lds, 5, P, F32, N, STREAM) == 0
            else:
                assert lib.spense_experts_linear_fp8b(h, P, K, P, lds, 5, None, P, 5, P, F32, N, STREAM) == 0
            assert (lib.host_seen8(X) == P) == want, (kind, lds)
        for lds in (1 << 23, 1 << 37, (1 << 62) + 5):
            st = (lib.spense_linear_fp8b(h, P, K, P, lds, 5, P, F32, N, STREAM) if kind == "codes" else
                  lib.spense_experts_linear_fp8b(h, P, K, P, lds, 5, None, P, 5, P, F32, N, STREAM))
            assert st == sdg.SPENSE_EUNSUPPORTED, (kind, lds)
        lib.spense_free(h)


def test_info(lib):
    i = sdg.LayerInfo()
    h = layer(lib)
    assert lib.spense_info(h, ctypes.byref(i)) == 0
    assert (i.split, i.N, i.K, i.K_d, i.N_s, i.N_d, i.wdtype) == (5, N, K, K, 1, N, FP8)
    assert i.weight_bytes == N * K + 4 * BLOCKS and i.device_bytes == N * K + 8 * BLOCKS
    lib.spense_free(h)
    h = experts(lib, 1, 300)
    assert lib.spense_info(h, ctypes.byref(i)) == 0
    assert (i.split, i.N, i.N_s, i.N_d) == (6, 300, 4, 150) and i.weight_bytes == 4 * (300 * K + 4 * 4 * BLOCKS)
    lib.spense_free(h)
