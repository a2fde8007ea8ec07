"""Which bits the sums of the fp8b products keep where large products cancel.

The inputs: unit scales (448 in every block of 128 x 128 and 1 x 128), products
+2^16 and -2^16 (256 x 256) that cancel within an eight or between two, and
small ones of 1, 2 or 4 beside them.

Every product is a whole number, and so is every sum of some of them, below 2^24
(four of 2^16 in each of four blocks, and the small ones), so fp32 holds it
whatever the order.  Sums that are kept in full are therefore exact, and a bf16
result of them is the exact sum rounded.

Codes into bf16 may lose 2^-10 of the largest magnitude of each eight
(oracle.dropped_bits_ref); the rounding to bf16 is 2^-8 of the result, which is
off by that already: |Y - ref| <= (1 + 2^-8) dropped + 2^-8 |ref|.  On a
gate/up layer with gate and up sums off by e_g and e_u see
test_gpu_fp8b_experts.py."""

import numpy as np
import pytest
import torch

import oracle
import sparse_dense_gemm_amd as sdg

from fp8b_util import assert_close, dev, f64

pytestmark = pytest.mark.gpu


def codes_of(v):
    return oracle.nearest_e4m3(v)


def operands(M, N, K, seed, places=0):
    """Values x [M, K], w [N, K]: in every block one eight (by `places`) with +-2^16 and small products beside it, and two
    products of +-2^16 in other eights."""
    rng, at = np.random.default_rng(seed), np.random.default_rng(places)
    x, w = np.zeros((M, K)), np.zeros((N, K))
    for b in range(0, K, 128):
        e = b + 8 * at.integers(0, 14)
        x[:, e:e + 2], w[:, e], w[:, e + 1] = 256.0, 256.0, -256.0      # cancel within the eight
        x[:, e + 2:e + 7] = rng.choice([-2.0, -1.0, 1.0, 2.0], (M, 5))  # beside them
        w[:, e + 2:e + 7] = rng.choice([-2.0, -1.0, 1.0, 2.0], (N, 5))
        x[:, [e + 8, b + 120]], w[:, e + 8], w[:, b + 120] = 256.0, 256.0, -256.0  # cancel, in different eights
        x[:, e + 9:e + 12] = 1.0
        w[:, e + 9:e + 12] = rng.choice([-2.0, 1.0, 4.0], (N, 3))
    x[:, 127::128] = 448.0  # a block's largest value, so that its scale is 1, times a zero
    w[::128, 126::128] = 448.0
    return x, w


def test_operands():
    x, w = operands(5, 300, 512, 1)
    q, s = oracle.fp8b_quantize_ref(x.astype(np.float32))
    assert (s == 1).all() and np.array_equal(oracle.fp8b_values_ref(q, s), x)
    q, s = oracle.fp8b_quantize_ref(w.astype(np.float32), 128)
    assert (s == 1).all() and np.array_equal(oracle.fp8b_values_ref(q, s, 128), w)
    assert (np.abs(x) @ np.abs(w).T).max() < 2.0 ** 24 and np.abs(x @ w.T).max() < 2.0 ** 16


@pytest.mark.parametrize("M,forced", [(1, None), (5, None), (29, None), (130, None), (600, None)]
                         + [(300, f"{c}") for c in range(5)])
def test_cancelling_products(M, forced, monkeypatch):
    N, K = 300, 512
    x, w = operands(M, N, K, M)
    ref = x @ w.T
    layer = sdg.SpenseLinearFp8b(dev(codes_of(w)), torch.ones((3, 4), device="cuda"))
    X = dev(x.astype(np.float32)).bfloat16()
    q, s = dev(codes_of(x)), torch.ones((M, 4), device="cuda")
    calls = {"bf16": lambda Y: layer(X, Y), "w8a8": lambda Y: layer.w8a8(X, Y), "codes": lambda Y: layer.quantized(q, s, Y)}
    for kind, call in calls.items():
        for yt in (torch.float32, torch.bfloat16):
            monkeypatch.delenv("SPENSE_FP8B", raising=False)
            if forced and not (forced == "4" and kind != "bf16" and yt == torch.float32):
                monkeypatch.setenv("SPENSE_FP8B", forced)
            Y = call(torch.empty((M, N), dtype=yt, device="cuda"))
            if kind == "bf16" or yt == torch.float32:
                want = dev(ref.astype(np.float32)).to(yt)  # ref is a number of fp32
                assert torch.equal(Y, want), (kind, yt, M, forced)
            else:
                tol = (1 + 2.0 ** -8) * oracle.dropped_bits_ref(x, w) + 2.0 ** -8 * np.abs(ref)
                assert_close(f64(Y), ref, tol, (kind, yt, M, forced))
    layer.close()


@pytest.mark.parametrize("M", [3, 150])
def test_cancelling_products_of_experts(M):
    E, N, K = 3, 300, 512
    x, _ = operands(M, N, K, 7)
    w = np.stack([operands(1, N, K, 8 + e)[1] for e in range(E)])
    ref = np.concatenate([x[e::E] @ w[e].T for e in range(E)])
    dropped = np.concatenate([oracle.dropped_bits_ref(x[e::E], w[e]) for e in range(E)])
    assert np.abs(ref).max() < 2.0 ** 24
    rows = np.concatenate([np.arange(M)[e::E] for e in range(E)]).astype(np.int32)
    off = np.concatenate([[0], np.cumsum([len(range(e, M, E)) for e in range(E)])]).astype(np.int32)
    h = sdg.SpenseExpertsFp8b(dev(codes_of(w)), torch.ones((E, 3, 4), device="cuda"))
    q, s = dev(codes_of(x)), torch.ones((M, 4), device="cuda")
    Y = h.quantized(q, s, dev(off), torch.empty((M, N), device="cuda"), rows=dev(rows))
    assert np.array_equal(f64(Y), ref)
    Y = h.quantized(q, s, dev(off), torch.empty((M, N), dtype=torch.bfloat16, device="cuda"), rows=dev(rows))
    assert_close(f64(Y), ref, (1 + 2.0 ** -8) * dropped + 2.0 ** -8 * np.abs(ref), "bf16")
    h.close()


def test_normal_inputs_lose_less_than_the_rounding():
    """The drop is at most 2^-15 of the results' rms (3.1e-5) on normal inputs, by the values that it rounds elsewhere.

    Rounded values differ from those of the full sums (fp32 Y) where a border lies between the two sums.  With a
    difference of rms 2^-15, its mean magnitude 0.8 2^-15 rms, and steps of bf16 of at least 2^-8 |y|, the share at a
    value y = z rms is at most min(1, a / |z|), a = 0.8 2^-7; over normal z that is 0.8 a (ln(1 / a) + 1.06) = 0.031."""
    M, N, K = 512, 1024, 4096
    g = torch.Generator("cuda").manual_seed(1)
    wc, ws = torch.empty((N, K), dtype=torch.uint8, device="cuda"), torch.empty((N // 128, K // 128), device="cuda")
    sdg.spense_quantize_fp8b(torch.randn(N, K, device="cuda", generator=g), wc, ws, rows=128)
    xc, xs = torch.empty((M, K), dtype=torch.uint8, device="cuda"), torch.empty((M, K // 128), device="cuda")
    sdg.spense_quantize_fp8b(torch.randn(M, K, device="cuda", generator=g), xc, xs)
    layer = sdg.SpenseLinearFp8b(wc, ws)
    full = layer.quantized(xc, xs, torch.empty((M, N), device="cuda"))
    Y = layer.quantized(xc, xs, torch.empty((M, N), dtype=torch.bfloat16, device="cuda"))
    assert (Y != full.bfloat16()).double().mean() < 0.031
    assert torch.equal(Y, layer.quantized(xc, xs, torch.empty_like(Y)))
    layer.close()
