"""The binding takes codes as bytes or e4m3fn numbers, and no other 8-bit floats:
their bytes stand for other numbers (tensors on the CPU: every refusal comes
before the library's call)."""

import pytest
import torch

import sparse_dense_gemm_amd as sdg

M, K, E, N = 4, 256, 2, 128
OTHERS = [t for t in ("float8_e5m2", "float8_e4m3fnuz", "float8_e5m2fnuz", "float8_e8m0fnu") if hasattr(torch, t)]


def calls(codes):
    s, X = torch.zeros((M, 2)), torch.zeros((M, K))
    off = torch.zeros(E + 1, dtype=torch.int32)
    W = codes[:1].expand(E * N, K).contiguous().view(E, N, K)
    return {
        "quantize": lambda: sdg.spense_quantize_fp8b(X, codes, s, stream=0),
        "dequantize": lambda: sdg.spense_dequantize_fp8b(codes, s, X, stream=0),
        "pack": lambda: sdg.spense_pack_fp8b(W[0], torch.zeros((1, 2)), stream=0),
        "pack experts": lambda: sdg.spense_pack_experts_fp8b(W, torch.zeros((E, 1, 2)), stream=0),
        "linear": lambda: sdg._linear_fp8b(1, sdg._Dims(K, N, 1), codes, s, torch.zeros((M, N)), None, 0),
        "experts": lambda: sdg._experts_linear_fp8b(1, sdg._Dims(K, N, E), codes, s, off, torch.zeros((M, N)), None, None, 0),
        "norm": lambda: sdg.spense_block_norm(X, None, None, codes, eps=1e-6, yscales=s, stream=0),
    }


@pytest.fixture
def library(monkeypatch):
    class Lib:
        def __getattr__(self, name):
            return lambda *a: 0

    monkeypatch.setattr(sdg, "_lib_handle", Lib())


@pytest.mark.parametrize("t", OTHERS)
@pytest.mark.parametrize("call", calls(torch.zeros((M, K), dtype=torch.uint8)))
def test_other_floats_are_refused(library, t, call):
    with pytest.raises(TypeError):
        calls(torch.zeros((M, K), dtype=torch.uint8).view(getattr(torch, t)))[call]()


@pytest.mark.parametrize("t", [torch.uint8, torch.float8_e4m3fn])
def test_codes_are_taken(library, t):
    for name, call in calls(torch.zeros((M, K), dtype=torch.uint8).view(t)).items():
        call()
