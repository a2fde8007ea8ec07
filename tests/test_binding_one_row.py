"""One row of a larger tensor, as the last position of a sequence is: its stride,
whatever it says, refuses nothing (the C calls recorded, tensors on the CPU)."""

import types

import pytest
import torch

import sparse_dense_gemm_amd as sdg

K, N = 256, 64
LONG = 1 << 23  # elements between positions: more than a row stride may be


@pytest.fixture
def calls(monkeypatch):
    """Arguments of the library's calls, all of which succeed."""
    seen = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.append((name, a)) or 0

    monkeypatch.setattr(sdg, "_lib_handle", Lib())
    return seen


def last(dtype, cols=K):
    """[1, cols] whose stride is LONG, and one whose stride is less than a row."""
    t = torch.zeros(2 * cols, dtype=dtype)
    return t.as_strided((1, cols), (LONG, 1)), t.as_strided((1, cols), (1, 1))


DIMS = sdg._Dims(K, N, 1)


def test_linear_layers(calls):
    layer = types.SimpleNamespace(handle=1, _dims=DIMS, _sizes=lambda X, Y: sdg.SpenseLinearFp8b._sizes(layer, X, Y))
    for X, Y in zip(last(torch.bfloat16), last(torch.float32, N)):
        for call in (sdg.SpenseLinearFp8b.__call__, sdg.SpenseLinearFp8b.w8a8):
            call(layer, X, Y, stream=0)
            name, a = calls.pop()
            assert K in a and N in a and LONG not in a, (name, a)
    for (q, Y) in zip(last(torch.uint8), last(torch.bfloat16, N)):
        for s in last(torch.float32, 2):
            sdg.SpenseLinearFp8b.quantized(layer, q, s, Y, stream=0)
            _, a = calls.pop()
            assert (a[2], a[4], a[8]) == (K, 2, N)


def test_experts(calls):
    off = torch.zeros(2, dtype=torch.int32)
    for X, Y in zip(last(torch.bfloat16), last(torch.float32, N)):
        sdg._experts_linear(1, DIMS, X, off, Y, None, sdg.DT_BF16, None, 0)
        assert LONG not in calls.pop()[1]
    for q, Y in zip(last(torch.uint8), last(torch.float32, N)):
        sdg._experts_linear_fp8b(1, DIMS, q, last(torch.float32, 2)[0], off, Y, None, None, 0)
        assert LONG not in calls.pop()[1]


def test_format(calls):
    for X, q in zip(last(torch.bfloat16), last(torch.uint8)):
        for s in last(torch.float32, 2):
            sdg.spense_quantize_fp8b(X, q, s, stream=0)
            sdg.spense_dequantize_fp8b(q, s, X, stream=0)
            (_, a), (_, b) = calls.pop(), calls.pop()
            assert (a[1], a[3], a[9]) == (K, 2, K) and (b[4], b[7], b[9]) == (K, K, 2)


@pytest.mark.parametrize("i", [0, 1])
def test_norm(calls, i):
    O, R, G = (last(torch.bfloat16)[i] for _ in range(3))
    q, s = last(torch.uint8)[i], last(torch.float32, 2)[i]
    sdg.spense_block_norm(O, R, R, q, gate=G, eps=1e-6, yscales=s, stream=0)
    call = sdg.NormCall.from_buffer_copy(calls.pop()[1][0])
    assert (call.T, call.H, call.ldo, call.ldr, call.ldro, call.ldy, call.lds) == (1, K, K, K, K, K, 2)
    wide = torch.zeros((1, K + 8), dtype=torch.bfloat16)  # the sum in the place of a wider row's beginning
    sdg.spense_block_norm(O, wide, wide[:, :K], None, eps=1e-6, stream=0)
    call = sdg.NormCall.from_buffer_copy(calls.pop()[1][0])
    assert call.ldr == call.ldro == K and call.residual == call.residual_out


def test_an_ordinary_stride_stays(calls):
    """A padded row's stride, which may be what lets it be read in place."""
    X = torch.zeros((1, 264), dtype=torch.bfloat16)[:, :K + 3]
    off = torch.zeros(2, dtype=torch.int32)
    sdg._experts_linear(1, DIMS, X, off, torch.zeros((1, N)), None, sdg.DT_BF16, None, 0)
    assert 264 in calls.pop()[1]
