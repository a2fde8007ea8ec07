"""Calls without rows, on empty tensors (which have no address), on the GPU."""

import pytest
import torch

import sparse_dense_gemm_amd as sdg

pytestmark = pytest.mark.gpu


def test_sum_over_no_rows_is_zero():
    pos = torch.zeros((5, 2), dtype=torch.int32, device="cuda")
    for yt in (torch.float32, torch.bfloat16):
        Y = torch.full((5, 7), 3.0, dtype=yt, device="cuda")
        sdg.spense_experts_combine(torch.empty((0, 7), device="cuda"), pos, torch.ones((5, 2), device="cuda"), Y)
        assert (Y == 0).all()


def test_no_rows_write_nothing():
    h = sdg.SpenseExperts(torch.zeros((2, 16, 32), dtype=torch.bfloat16, device="cuda"))
    offsets = torch.zeros(3, dtype=torch.int32, device="cuda")
    Y = torch.full((4, 16), 5.0, device="cuda")
    X = torch.zeros((4, 32), dtype=torch.bfloat16, device="cuda")
    h(X, offsets, Y[:0])
    h(X[:0], offsets, Y[:0], rows=torch.empty(0, dtype=torch.int32, device="cuda"))
    h(X, offsets, Y)                        # rows, but of no expert
    e, u8 = torch.empty((0, 32), device="cuda"), dict(dtype=torch.uint8, device="cuda")
    sdg.spense_quantize_mx4(e, torch.empty((0, 16), **u8), torch.empty((0, 1), **u8))
    sdg.spense_dequantize_mx4(torch.empty((0, 16), **u8), torch.empty((0, 1), **u8), e)
    torch.cuda.synchronize()
    assert (Y == 5.0).all()
