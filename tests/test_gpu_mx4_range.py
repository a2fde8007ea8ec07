"""The top of the exponents' range in products with mx4 weights, and activations
that are not finite.  With bf16 activations a weight of 2^128 or more (scale bytes
253 and 254 only) is an infinity; with mx4 activations all are as they are."""

import numpy as np
import pytest
import torch

import oracle
import sparse_dense_gemm_amd as sdg
from test_gpu_mx4 import dev, tolerance

pytestmark = pytest.mark.gpu

N, K = 48, 192


def layers(codes, scales):
    """The same weights as a linear layer and as the second of two experts: run(X, mx4 activations) -> Y."""
    lin = sdg.SpenseLinearMx4(dev(codes), dev(scales), K=K)
    ex = sdg.SpenseExperts(dev(np.stack([codes, codes])), sdg.DT_MX4, scales=dev(np.stack([scales, scales])), K=K)

    def linear(X, a4):
        Y = torch.empty((X.shape[0], N), device="cuda")
        return (lin.w4a4 if a4 else lin)(X, Y)

    def experts(X, a4):
        Y = torch.empty((X.shape[0], N), device="cuda")
        off = dev(np.array([0, 0, X.shape[0]], dtype=np.int32))
        return ex(X, off, Y, adtype=sdg.DT_MX4 if a4 else sdg.DT_BF16)

    return linear, experts


def test_weights_at_the_top_of_the_range():
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    scales = rng.integers(240, 253, (N, K // 32)).astype(np.uint8)
    scales[::3] = 252                                     # the largest that holds every code in bf16
    big = np.zeros(N, dtype=bool)
    big[1::4] = True                                      # rows with a block at 253 or 254
    scales[1::8, 2], scales[5::8, 3] = 253, 254
    codes[1::8, 32] = 0x67                                # 6 and 4 times 2^126: past 2^128
    codes[5::8, 48] = 0x74                                # 2 and 6 times 2^127
    W = oracle.mx4_values_ref(codes, scales, K)
    x = np.exp2(rng.integers(-60, -50, (20, K))) * rng.choice([-1.0, 1.0], (20, K))
    X = dev(x.astype(np.float32)).bfloat16()
    for run in layers(codes, scales):
        ref, B = oracle.product_ref(oracle.mx4_values_ref(*oracle.mx4_quantize_ref(x), K), W)
        y = run(X, True).cpu().numpy().astype(np.float64)
        assert (np.abs(y - ref) <= tolerance(K, B, ref, False)).all()
        ref, B = oracle.product_ref(x, W)
        y = run(X, False).cpu().numpy().astype(np.float64)
        assert (np.abs(y - ref) <= tolerance(K, B, ref, False))[:, ~big].all()
        assert not np.isfinite(y[:, big]).any()


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_an_activation_that_is_not_finite(bad):
    """Its own row only, and all of that row where no weight beside it is zero."""
    rng = np.random.default_rng(2)
    codes = rng.choice([1, 2, 3, 5, 9, 10, 15], (N, K)).astype(np.uint8)
    codes = codes[:, ::2] | (codes[:, 1::2] << 4)
    scales = rng.integers(120, 130, (N, K // 32)).astype(np.uint8)
    x = rng.standard_normal((20, K)).astype(np.float32)
    x[7, 70] = bad
    X = dev(x).bfloat16()
    for run in layers(codes, scales):
        for a4 in (False, True):
            y = run(X, a4).cpu().numpy()
            assert not np.isfinite(y[7]).any(), a4
            assert np.isfinite(np.delete(y, 7, 0)).all(), a4
