"""Which bits the sums of spense_linear_w8a8 on an input-split layer keep where
large products cancel: at most 2^-10 of the sum of the products' magnitudes is
lost, and nothing by spense_linear on the same layer.

The operands are those of test_gpu_fp8b_sums.py with one token scale (the largest
value 448 meets a zero weight), whole numbers whose sums fp32 holds exactly."""

import numpy as np
import pytest
import torch

import sparse_dense_gemm_amd as sdg
from test_gpu_fp8b_sums import codes_of, operands

from fp8b_util import assert_close, dev, f64

pytestmark = pytest.mark.gpu

N, K = 256, 1024


@pytest.mark.parametrize("M", [1, 4, 64, 512])
@pytest.mark.parametrize("form", ["dense columns", "2:4"])
def test_cancelling_products(M, form):
    x, w = operands(M, N, K, 3)
    w[::128, 126::128] = 0.0
    if form == "2:4":  # the two largest of four are all there is
        four = w.reshape(N, K // 4, 4)
        keep = np.zeros_like(four)
        np.put_along_axis(keep, np.argsort(-np.abs(four), 2, kind="stable")[..., :2], 1.0, 2)
        w = (four * keep).reshape(N, K)
    ref, mags = x @ w.T, np.abs(x) @ np.abs(w).T
    assert mags.max() < 2.0 ** 24
    h = sdg.spense_pack(dev(codes_of(w)), sdg.DT_FP8, scales=torch.ones(N, device="cuda"),
                        dense_cols=np.arange(K if form == "dense columns" else 0))
    X = dev(x.astype(np.float32)).bfloat16()
    Y = torch.empty((M, N), device="cuda")
    sdg.spense_linear(h, X, Y)
    assert np.array_equal(f64(Y), ref)
    for yt in (torch.float32, torch.bfloat16):
        Y = torch.empty((M, N), dtype=yt, device="cuda")
        sdg.spense_linear_w8a8(h, X, Y)
        rounding = (2.0 ** -8 if yt == torch.bfloat16 else 0.0) * (np.abs(ref) + 2.0 ** -10 * mags)
        assert_close(f64(Y), ref, 2.0 ** -10 * mags + rounding, (M, form, yt))
        Z = torch.empty_like(Y)
        sdg.spense_linear_w8a8(h, X, Z)
        assert torch.equal(Y, Z)
    sdg.spense_free(h)
