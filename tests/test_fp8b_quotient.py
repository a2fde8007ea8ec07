"""The quotients of the fp8b codes and scales (spense_quotient.h), compiled for the
host: the same bits as a division, from any reciprocal within a unit in the last
place, for every significand that does not divide."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import host_library as hl
import oracle

ALL = (1 << 23) - 1


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir(os.path.join(hl.ROCM, "include", "hip")):
        pytest.skip("needs g++ and the HIP headers")
    out = os.path.join(str(tmp_path_factory.mktemp("quotient")), "libquotient.so")
    # no contraction: the product and the sums are rounded as they are written
    r = subprocess.run([gxx, "-std=c++17", "-O2", "-ffp-contract=off", "-w", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__",
                        f"-I{hl.ROCM}/include", os.path.join(hl.HERE, "quotient_host.cpp"), "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    lib = ctypes.CDLL(out)
    u32, i64, f = ctypes.c_uint32, ctypes.c_int64, ctypes.c_float
    lib.host_by_reciprocal.argtypes = [f]
    lib.host_wrong_reciprocals.argtypes = [ctypes.c_int, u32, u32, ctypes.c_int, ctypes.POINTER(u32)]
    lib.host_wrong_quotients.argtypes = [ctypes.c_int, u32, u32, ctypes.c_void_p, ctypes.c_int, ctypes.c_int]
    lib.host_wrong_scales.argtypes = [ctypes.c_int, u32]
    for n in ("reciprocals", "quotients", "scales"):
        getattr(lib, f"host_wrong_{n}").restype = i64
    return lib


def borders():
    v = oracle.e4m3_values()[:127]
    return np.ascontiguousarray(((v[1:] + v[:-1]) / 2).astype(np.float32))


@pytest.mark.parametrize("e", [-90, 1, 99])
def test_every_significand(lib, e):
    which = ctypes.c_uint32()
    assert lib.host_wrong_reciprocals(e, 0, 1, 0, ctypes.byref(which)) == 0, which.value
    # the one that is turned away is the one that goes wrong
    assert lib.host_wrong_reciprocals(e, 0, 1, 1, ctypes.byref(which)) == 1 and which.value == ALL


@pytest.mark.parametrize("e", [-90, -1, 0, 99])
def test_quotients_at_the_borders_of_codes(lib, e):
    b = borders()
    for first, step in ((0, 4093), (1, 1 << 20), (ALL - 64, 1)):
        assert lib.host_wrong_quotients(e, first, step, b.ctypes.data, len(b), 0) == 0, (e, first)
    assert lib.host_wrong_quotients(e, ALL, 1, b.ctypes.data, len(b), 1) > 0


@pytest.mark.parametrize("e", [-80, 0, 8, 127])
def test_scales(lib, e):
    assert lib.host_wrong_scales(e, 1) == 0


def test_which_scales_divide(lib):
    for s, want in ((1.0, 1), (2.0 ** -90, 1), (2.0 ** 100, 1), (2.0 ** -90 * (1 - 2.0 ** -24), 0),
                    (2.0 ** 100 * (1 + 2.0 ** -23), 0), (2 - 2.0 ** -23, 0), (1.5 - 2.0 ** -23, 1), (2 - 2.0 ** -22, 1),
                    (float("nan"), 0), (float("inf"), 0), (0.0, 0)):
        assert bool(lib.host_by_reciprocal(s)) == bool(want), s
