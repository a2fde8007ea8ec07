"""Refusals of the fp8b and block-norm entry points: every bad argument is
rejected on the host before any HIP call (so these run without a GPU), and the
binding refuses tensors that do not hold what the call would read or write."""

import ctypes

import pytest
import torch

import sparse_dense_gemm_amd as sdg

P = 1 << 20  # never dereferenced: validation fails before any HIP call
OK, EINVAL, EUNSUP = sdg.SPENSE_OK, sdg.SPENSE_EINVAL, sdg.SPENSE_EUNSUPPORTED
F32, BF16, FP8, MX4 = sdg.DT_F32, sdg.DT_BF16, sdg.DT_FP8, sdg.DT_MX4
BIG = (1 << 24) + 1


def quantize(X=P, t=F32, M=4, K=300, ldx=300, rows=1, codes=P, ldc=300, scales=P, lds=3):
    return sdg._lib().spense_quantize_fp8b(X, t, M, K, ldx, rows, codes, ldc, scales, lds, None)


@pytest.mark.parametrize("kw,want", [
    (dict(X=None), EINVAL), (dict(codes=None), EINVAL), (dict(scales=None), EINVAL), (dict(M=-1), EINVAL),
    (dict(M=BIG), EINVAL), (dict(K=0), EINVAL), (dict(K=(1 << 20) + 1, ldx=1 << 21, ldc=1 << 21, lds=1 << 14), EINVAL),
    (dict(ldx=299), EINVAL), (dict(ldc=299), EINVAL), (dict(lds=2), EINVAL), (dict(rows=0), EINVAL),
    (dict(rows=64), EINVAL), (dict(t=9), EINVAL), (dict(t=FP8), EUNSUP), (dict(t=MX4), EUNSUP), (dict(M=0), OK),
    (dict(M=0, X=None, codes=None, scales=None), OK),
])
def test_quantize_rejects(kw, want):
    assert quantize(**kw) == want


def dequantize(codes=P, ldc=300, scales=P, lds=3, rows=128, M=4, K=300, Y=P, t=F32, ldy=300):
    return sdg._lib().spense_dequantize_fp8b(codes, ldc, scales, lds, rows, M, K, Y, t, ldy, None)


@pytest.mark.parametrize("kw,want", [
    (dict(codes=None), EINVAL), (dict(scales=None), EINVAL), (dict(Y=None), EINVAL), (dict(M=-1), EINVAL),
    (dict(K=0), EINVAL), (dict(ldy=299), EINVAL), (dict(ldc=299), EINVAL), (dict(lds=2), EINVAL),
    (dict(rows=2), EINVAL), (dict(t=-1), EINVAL), (dict(t=FP8), EUNSUP), (dict(t=MX4), EUNSUP), (dict(M=0), OK),
])
def test_dequantize_rejects(kw, want):
    assert dequantize(**kw) == want


def pack(codes=P, ldc=300, scales=P, lds=3, N=16, K=300, out=True):
    h = ctypes.c_void_p()
    st = sdg._lib().spense_pack_fp8b(codes, ldc, scales, lds, N, K, None, ctypes.byref(h) if out else None)
    assert not h.value
    return st


@pytest.mark.parametrize("kw", [dict(codes=None), dict(scales=None), dict(N=0), dict(N=BIG), dict(K=0), dict(ldc=299),
                                dict(lds=2), dict(out=False)])
def test_pack_rejects(kw):
    assert pack(**kw) == EINVAL


def pack_experts(W=P, scales=P, E=4, N=16, K=300, ldw=300, lds=3, glu=0, out=True):
    h = ctypes.c_void_p()
    st = sdg._lib().spense_pack_experts_fp8b(W, scales, E, N, K, ldw, lds, glu, None, ctypes.byref(h) if out else None)
    assert not h.value
    return st


@pytest.mark.parametrize("kw", [dict(W=None), dict(scales=None), dict(E=0), dict(E=1025), dict(N=0), dict(K=0),
                                dict(ldw=299), dict(lds=2), dict(glu=1, N=15), dict(out=False)])
def test_pack_experts_rejects(kw):
    assert pack_experts(**kw) == EINVAL


def test_null_handles():
    lib = sdg._lib()
    assert lib.spense_linear_fp8b(None, P, 300, P, 3, 1, P, F32, 16, None) == EINVAL
    assert lib.spense_experts_linear_fp8b(None, P, 300, P, 3, 1, None, P, 1, P, F32, 16, None) == EINVAL


def norm(**kw):
    """A call that would run (T = 0) unless something is wrong."""
    args = dict(T=0, H=300, O=P, ldo=300, O_rows=0, pos=None, weights=None, post=P, pre=P, gate=P, ldg=0, residual=P,
                ldr=300, residual_out=P, ldro=300, Y=P, ldy=300, yscales=None, lds=0, k=0, otype=F32, wtype=BF16,
                gtype=F32, rtype=BF16, ytype=BF16, scale=1.0, eps=1e-6)
    args.update(kw)
    return sdg._lib().spense_block_norm(ctypes.byref(sdg.NormCall(**args)), None)


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(T=-1), EINVAL), (dict(T=BIG), EINVAL), (dict(H=0), EINVAL), (dict(H=(1 << 20) + 1), EINVAL),
    (dict(T=1, O=None), EINVAL), (dict(T=1, Y=None, residual_out=None), EINVAL),
    (dict(Y=None, residual_out=None), OK), (dict(eps=0.0), EINVAL),
    (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(eps=float("inf")), EINVAL),
    (dict(eps=1e-40), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(scale=float("nan")), EINVAL),
    (dict(ldo=299), EINVAL), (dict(ldg=299), EINVAL), (dict(ldg=-300), EINVAL), (dict(ldr=299), EINVAL),
    (dict(ldro=299), EINVAL), (dict(ldy=299), EINVAL), (dict(ldro=301), EINVAL),  # in place with another stride
    (dict(residual=P + 4096, ldro=301), OK),
    (dict(pos=P), EINVAL), (dict(weights=P), EINVAL), (dict(pos=P, weights=P, k=0), EINVAL),
    (dict(pos=P, weights=P, k=1025), EINVAL), (dict(pos=P, weights=P, k=2, O_rows=-1), EINVAL),
    (dict(pos=P, weights=P, k=2, O_rows=BIG), EINVAL), (dict(pos=P, weights=P, k=2), OK),
    (dict(yscales=P), EINVAL), (dict(T=1, ytype=FP8), EINVAL), (dict(ytype=FP8), EINVAL), (dict(ytype=FP8, yscales=P, lds=2), EINVAL),
    (dict(ytype=FP8, yscales=P, lds=3), OK), (dict(otype=FP8), EUNSUP), (dict(otype=7), EINVAL),
    (dict(wtype=MX4), EUNSUP), (dict(gtype=FP8), EUNSUP), (dict(rtype=FP8), EUNSUP), (dict(ytype=MX4), EUNSUP),
    (dict(gate=None, gtype=9, ldg=-5), OK), (dict(residual=None, ldr=0), OK), (dict(Y=None, ldy=0, ytype=9), OK),
    (dict(post=None, pre=None, wtype=9), OK), (dict(Y=None, ytype=9, yscales=P), EINVAL),
])
def test_block_norm_rejects(kw, want):
    assert norm(**kw) == want


OTHER = {name: P + (i << 16) for i, name in enumerate(("O", "post", "pre", "gate", "residual", "residual_out", "Y"))}


@pytest.mark.parametrize("out,into", [("Y", "O"), ("Y", "post"), ("Y", "pre"), ("Y", "gate"), ("Y", "residual"),
                                      ("Y", "residual_out"), ("residual_out", "O"), ("residual_out", "gate")])
def test_block_norm_refuses_outputs_in_place(out, into):
    assert norm(**{**OTHER, "T": 0, out: OTHER[into]}) == OK
    assert norm(**{**OTHER, "T": 3, out: OTHER[into]}) == EINVAL


def test_packed_call_is_the_structure():
    """The binding's packing of a call has the bytes of the C structure."""
    values = (*range(1, 26), 0.5, 0.25)
    assert bytes(sdg.NormCall(*values)) == sdg._NORM.pack(*values)


def test_block_norm_null():
    assert sdg._lib().spense_block_norm(None, None) == EINVAL


# ---- the binding (tensors on the CPU: every refusal comes before the library's call) ----

C, S, X = torch.zeros((4, 300), dtype=torch.uint8), torch.zeros((4, 3)), torch.zeros((4, 300))


@pytest.mark.parametrize("codes,scales", [
    (C[:3], S), (C, S[:3]), (C[:, :299], S), (C, S[:, :2]), (C.t().contiguous().t(), S), (C.int(), S), (C, S.double()),
    (C, S.bfloat16())])
def test_binding_checks_matrices(codes, scales):
    for call in (lambda: sdg.spense_quantize_fp8b(X, codes, scales, stream=0),
                 lambda: sdg.spense_dequantize_fp8b(codes, scales, X, stream=0)):
        with pytest.raises((ValueError, TypeError)):
            call()


def test_binding_checks_blocks():
    with pytest.raises(ValueError):
        sdg.spense_pack_fp8b(torch.zeros((129, 300), dtype=torch.uint8), torch.zeros((1, 3)), stream=0)
    W = torch.zeros((2, 260, 300), dtype=torch.uint8)
    for blocks, glu in ((2, False), (3, True), (5, True)):  # 260 rows: 3 blocks, or 2 of gate and 2 of up
        with pytest.raises(ValueError):
            sdg.spense_pack_experts_fp8b(W, torch.zeros((2, blocks, 3)), glu=glu, stream=0)
    with pytest.raises(ValueError):
        sdg.spense_pack_experts_fp8b(W, torch.zeros((1, 3, 3)), stream=0)
    with pytest.raises(ValueError):
        sdg.spense_pack_experts_fp8b(W.transpose(1, 2), torch.zeros((2, 3, 3)), stream=0)
    with pytest.raises(sdg.SpenseError):
        sdg.spense_quantize_fp8b(X, C, S, rows=3, stream=0)


def norm_call(**kw):
    H, T = 300, 4
    args = dict(O=torch.zeros((T, H)), residual=torch.zeros((T, H)), residual_out=torch.zeros((T, H)),
                Y=torch.zeros((T, H)), pre=torch.zeros(H), eps=1e-6, stream=0)
    args.update(kw)
    sdg.spense_block_norm(args.pop("O"), args.pop("residual"), args.pop("residual_out"), args.pop("Y"), **args)


@pytest.mark.parametrize("kw", [
    dict(residual=torch.zeros((3, 300))), dict(residual=torch.zeros((4, 299))), dict(residual_out=torch.zeros((4, 299))),
    dict(residual_out=torch.zeros((4, 300), dtype=torch.bfloat16)), dict(Y=torch.zeros((3, 300))),
    dict(pre=torch.zeros(299)), dict(post=torch.zeros(300, dtype=torch.bfloat16)), dict(gate=torch.zeros((3, 300))),
    dict(gate=torch.zeros((4, 299))), dict(gate=torch.zeros(299)), dict(pos=torch.zeros((4, 2), dtype=torch.int32)),
    dict(weights=torch.zeros((4, 2))), dict(pos=torch.zeros((4, 2)), weights=torch.zeros((4, 2))),
    dict(pos=torch.zeros((4, 2), dtype=torch.int32), weights=torch.zeros((4, 1))),
    dict(Y=C, yscales=torch.zeros((4, 2))), dict(Y=C, yscales=torch.zeros((4, 3), dtype=torch.float64)),
    dict(O=torch.zeros((4, 300), dtype=torch.float16)), dict(O=torch.zeros((300, 4)).t())])
def test_binding_checks_norm(kw):
    with pytest.raises((ValueError, TypeError)):
        norm_call(**kw)


def test_binding_refuses_codes_without_scales():
    with pytest.raises(sdg.SpenseError):
        norm_call(Y=C)
