"""Refusals of the mx4, experts' and router entry points: every bad argument
is rejected on the host before any HIP call (so these run without a GPU)."""

import ctypes

import pytest
import torch

import sparse_dense_gemm_amd as sdg

P = 1 << 20  # never dereferenced: validation fails before any HIP call
OK, EINVAL, EUNSUP = sdg.SPENSE_OK, sdg.SPENSE_EINVAL, sdg.SPENSE_EUNSUPPORTED
F32, BF16, FP8, MX4 = sdg.DT_F32, sdg.DT_BF16, sdg.DT_FP8, sdg.DT_MX4


def quantize(X=P, t=F32, M=4, K=64, ldx=64, codes=P, ldc=32, scales=P, lds=2):
    return sdg._lib().spense_quantize_mx4(X, t, M, K, ldx, codes, ldc, scales, lds, None)


@pytest.mark.parametrize("kw,want", [
    (dict(X=None), EINVAL), (dict(codes=None), EINVAL), (dict(scales=None), EINVAL),
    (dict(M=-1), EINVAL), (dict(M=(1 << 24) + 1), EINVAL), (dict(K=0), EINVAL), (dict(K=(1 << 20) + 1, ldx=1 << 21), EINVAL),
    (dict(ldx=63), EINVAL), (dict(ldc=31), EINVAL), (dict(lds=1), EINVAL),
    (dict(K=63, ldc=31), EINVAL), (dict(t=9), EINVAL), (dict(t=FP8), EUNSUP), (dict(t=MX4), EUNSUP),
    (dict(M=0), OK),  # nothing to do: no launch
])
def test_quantize_rejects(kw, want):
    assert quantize(**kw) == want


def dequantize(codes=P, ldc=32, scales=P, lds=2, M=4, K=64, Y=P, t=F32, ldy=64):
    return sdg._lib().spense_dequantize_mx4(codes, ldc, scales, lds, M, K, Y, t, ldy, None)


@pytest.mark.parametrize("kw,want", [
    (dict(codes=None), EINVAL), (dict(scales=None), EINVAL), (dict(Y=None), EINVAL), (dict(M=-1), EINVAL),
    (dict(K=0), EINVAL), (dict(ldy=63), EINVAL), (dict(ldc=31), EINVAL), (dict(lds=1), EINVAL), (dict(t=-1), EINVAL),
    (dict(t=FP8), EUNSUP), (dict(t=MX4), EUNSUP), (dict(M=0), OK),
])
def test_dequantize_rejects(kw, want):
    assert dequantize(**kw) == want


def pack_mx4(codes=P, ldc=32, scales=P, lds=2, N=16, K=64, out=True):
    h = ctypes.c_void_p()
    st = sdg._lib().spense_pack_mx4(codes, ldc, scales, lds, N, K, None, ctypes.byref(h) if out else None)
    assert not h.value
    return st


@pytest.mark.parametrize("kw", [dict(codes=None), dict(scales=None), dict(N=0), dict(N=(1 << 24) + 1), dict(K=0),
                                dict(ldc=31), dict(lds=1), dict(out=False)])
def test_pack_mx4_rejects(kw):
    assert pack_mx4(**kw) == EINVAL


def pack_experts(W=P, t=BF16, scales=None, E=4, N=16, K=64, ldw=64, lds=0, glu=0, out=True):
    h = ctypes.c_void_p()
    st = sdg._lib().spense_pack_experts(W, t, scales, E, N, K, ldw, lds, glu, None, ctypes.byref(h) if out else None)
    assert not h.value
    return st


@pytest.mark.parametrize("kw,want", [
    (dict(W=None), EINVAL), (dict(E=0), EINVAL), (dict(E=1025), EINVAL), (dict(N=0), EINVAL), (dict(K=0), EINVAL),
    (dict(ldw=63), EINVAL), (dict(scales=P), EINVAL), (dict(glu=1, N=15), EINVAL), (dict(t=17), EINVAL),
    (dict(out=False), EINVAL), (dict(t=F32), EUNSUP), (dict(t=FP8), EUNSUP),
    (dict(t=MX4, ldw=32), EINVAL), (dict(t=MX4, scales=P, ldw=31, lds=2), EINVAL),
    (dict(t=MX4, scales=P, ldw=32, lds=1), EINVAL),
])
def test_pack_experts_rejects(kw, want):
    assert pack_experts(**kw) == want


def test_null_handles():
    lib = sdg._lib()
    assert lib.spense_linear_w4a4(None, P, 1, 64, P, F32, 16, None) == EINVAL
    assert lib.spense_experts_linear(None, P, BF16, 1, 64, None, P, 1, P, F32, 16, None) == EINVAL


def route(logits=P, t=F32, T=20000, E=8, ldl=8, k=2, ids=P, weights=P, offsets=P, rows=P, pos=P, work=P):
    return sdg._lib().spense_route(logits, t, T, E, ldl, k, 1, ids, weights, offsets, rows, pos, work, None)


@pytest.mark.parametrize("kw,want", [
    (dict(logits=None), EINVAL), (dict(ids=None), EINVAL), (dict(weights=None), EINVAL), (dict(offsets=None), EINVAL),
    (dict(rows=None), EINVAL), (dict(pos=None), EINVAL), (dict(work=None), EINVAL), (dict(work=P + 2), EINVAL),
    (dict(T=-1), EINVAL), (dict(E=0), EINVAL), (dict(E=1025, ldl=1025), EINVAL), (dict(ldl=7), EINVAL),
    (dict(k=0), EINVAL), (dict(k=9), EINVAL), (dict(T=1 << 24, k=2), EINVAL), (dict(t=5), EINVAL),
    (dict(t=FP8), EUNSUP), (dict(t=MX4), EUNSUP),
])
def test_route_rejects(kw, want):
    assert route(**kw) == want


def test_route_workspace():
    lib = sdg._lib()
    assert lib.spense_route_workspace(1, 8, 2) == 0 and lib.spense_route_workspace(64, 8, 2) == 0
    assert lib.spense_route_workspace(100000, 128, 8) > 0
    # enough for every smaller number of tokens
    for E in (3, 128, 1000):
        sizes = [lib.spense_route_workspace(T, E, 2) for T in list(range(0, 3000)) + list(range(3000, 300000, 997))]
        assert sizes == sorted(sizes)
    for T, E, k in ((-1, 8, 2), (1, 0, 1), (1, 8, 9), (1, 2000, 1)):
        assert lib.spense_route_workspace(T, E, k) == EINVAL
        with pytest.raises(sdg.SpenseError):
            sdg.spense_route_workspace(T, E, k)


def combine(O=P, ot=F32, R=4, ldo=8, pos=P, w=P, T=2, k=2, N=8, Y=P, yt=F32, ldy=8):
    return sdg._lib().spense_experts_combine(O, ot, R, ldo, pos, w, T, k, N, Y, yt, ldy, None)


@pytest.mark.parametrize("kw,want", [
    (dict(O=None), EINVAL), (dict(pos=None), EINVAL), (dict(w=None), EINVAL), (dict(Y=None), EINVAL),
    (dict(R=-1), EINVAL), (dict(T=-1), EINVAL), (dict(k=0), EINVAL), (dict(N=0), EINVAL), (dict(ldo=7), EINVAL),
    (dict(ldy=7), EINVAL), (dict(ot=11), EINVAL), (dict(yt=11), EINVAL), (dict(ot=FP8), EUNSUP), (dict(yt=MX4), EUNSUP),
    (dict(T=0), OK),
])
def test_combine_rejects(kw, want):
    assert combine(**kw) == want


def test_binding_checks_shapes():
    """The binding refuses tensors that do not hold what the call would read or write."""
    x = torch.zeros((4, 64))
    c, s = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8)
    for codes, scales in ((c[:3], s), (c, s[:3]), (c[:, :31], s), (c, s[:, :1]), (c.t().contiguous().t(), s),
                          (c.int(), s)):
        with pytest.raises(ValueError):
            sdg.spense_quantize_mx4(x, codes, scales, stream=0)
        with pytest.raises(ValueError):
            sdg.spense_dequantize_mx4(codes, scales, x, stream=0)
        with pytest.raises(ValueError):
            sdg.spense_pack_mx4(codes, scales, N=4, K=64, stream=0)
    w = torch.zeros((3, 16, 64), dtype=torch.bfloat16)
    for bad in (w[:, :8], w.transpose(1, 2), w[0]):
        with pytest.raises((ValueError, IndexError)):
            sdg.spense_pack_experts(bad, stream=0)
    i = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError):
        sdg.spense_route(torch.zeros((4, 8)), 2, i, torch.zeros(8), torch.zeros(8, dtype=torch.int32), i, i, stream=0)
    with pytest.raises(ValueError):
        sdg.spense_route(torch.zeros((400, 8)), 1, *(torch.zeros(400, dtype=torch.int32) for _ in range(5)), stream=0)
