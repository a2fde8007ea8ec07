"""GPU tests of the fp8b calls and of the block norm where sizes and offsets are
large: weights that are streamed past the caches, rows further apart than 31 bits
of elements, more threads than one launch takes.

Products are compared with the oracle within the tolerances of fp8b_util.py, calls
on far rows bit for bit with the same call on dense copies."""

import numpy as np
import pytest
import torch

import oracle
import sparse_dense_gemm_amd as sdg

from fp8b_util import assert_close, f64, product_tolerance

pytestmark = pytest.mark.gpu

FAR = (1 << 30) + 8  # elements between rows: the third row starts past 2^31


def far(M, K, ld, dtype, fill=None):
    """An [M, K] matrix with rows ld apart; what lies between them is not touched."""
    t = torch.empty(((M - 1) * ld + K,), dtype=dtype, device="cuda").as_strided((M, K), (ld, 1))
    if fill is not None:
        t.copy_(fill)
    return t


@pytest.fixture(scope="module")
def streamed():
    """A layer of more than 96 MiB, with its sampled columns' weights."""
    N, K = 20005, 5000
    g = torch.Generator("cuda").manual_seed(11)
    c = torch.empty((N, K), dtype=torch.uint8, device="cuda")
    s = torch.empty((-(-N // 128), -(-K // 128)), device="cuda")
    sdg.spense_quantize_fp8b(0.02 * torch.randn(N, K, device="cuda", generator=g), c, s, rows=128)
    layer = sdg.SpenseLinearFp8b(c, s)
    assert layer.info["device_bytes"] > 96 << 20
    n = np.r_[0:17, 125:131, 10000:10008, N - 9:N]
    W = oracle.e4m3_values()[c[n].cpu().numpy()] * np.repeat(s.double().cpu().numpy()[n // 128], 128, 1)[:, :K]
    yield layer, n, W, N, K
    layer.close()


@pytest.mark.parametrize("kind", ["bf16", "w8a8", "codes"])
@pytest.mark.parametrize("M,forced", [(13, "0"), (13, "1"), (13, "2"), (1, None), (16, None), (29, None), (33, None),
                                      (64, None), (65, None)])
def test_streamed_weights(streamed, kind, M, forced, monkeypatch):
    layer, n, W, N, K = streamed
    if forced:
        monkeypatch.setenv("SPENSE_FP8B", forced)
    X = torch.randn(M, K, device="cuda", generator=torch.Generator("cuda").manual_seed(M)).bfloat16()
    xq, xs = torch.empty((M, K), dtype=torch.uint8, device="cuda"), torch.empty((M, -(-K // 128)), device="cuda")
    sdg.spense_quantize_fp8b(X, xq, xs)
    x = f64(X) if kind == "bf16" else oracle.fp8b_values_ref(xq.cpu().numpy(), xs.cpu().numpy())
    ref, B = oracle.product_ref(x, W)
    for yt in (torch.float32, torch.bfloat16):
        Y = torch.full((M, N), float("nan"), dtype=yt, device="cuda")
        if kind == "bf16":
            layer(X, Y)
        elif kind == "w8a8":
            layer.w8a8(X, Y)
        else:
            layer.quantized(xq, xs, Y)
        assert_close(f64(Y[:, n]), ref, product_tolerance(x, W, ref, B, K, kind != "bf16", yt), (kind, M, forced, yt))
        assert not Y.isnan().any()


def test_quantize_far_rows():
    M, K = 3, 300
    x = torch.randn(M, K, device="cuda").bfloat16()
    for rows in (1, 128):
        c, s = torch.empty((M, K), dtype=torch.uint8, device="cuda"), torch.empty((-(-M // rows), 3), device="cuda")
        sdg.spense_quantize_fp8b(x, c, s, rows=rows)
        C, S = far(M, K, FAR, torch.uint8), far(s.shape[0], 3, FAR, torch.float32)
        sdg.spense_quantize_fp8b(far(M, K, FAR, torch.bfloat16, x), C, S, rows=rows)
        assert torch.equal(C, c) and torch.equal(S, s)
        y = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
        Y = far(M, K, FAR, torch.bfloat16)
        sdg.spense_dequantize_fp8b(c, s, y, rows=rows)
        sdg.spense_dequantize_fp8b(C, S, Y, rows=rows)
        assert torch.equal(Y, y)


@pytest.mark.parametrize("picked", [False, True])
def test_norm_far_rows(picked):
    T, H = 3, 520
    g = torch.Generator("cuda").manual_seed(1)
    O, R = (torch.randn(T, H, device="cuda", generator=g).bfloat16() for _ in range(2))
    w, gate = torch.rand(H, device="cuda", generator=g), torch.rand(T, H, device="cuda", generator=g).bfloat16()
    kw = dict(pre=w, post=w, eps=1e-6, scale=0.5)
    if picked:
        kw.update(pos=torch.tensor([[2, 0], [1, 2], [2, 2]], dtype=torch.int32, device="cuda"),
                  weights=torch.rand(T, 2, device="cuda", generator=g))
    r, q, s = torch.empty_like(R), torch.empty((T, H), dtype=torch.uint8, device="cuda"), torch.empty((T, 5), device="cuda")
    sdg.spense_block_norm(O, R, r, q, gate=gate, yscales=s, **kw)
    B = torch.bfloat16
    r2, q2, s2 = far(T, H, FAR, B, R), far(T, H, FAR, torch.uint8), far(T, 5, FAR, torch.float32)
    sdg.spense_block_norm(far(T, H, FAR, B, O), r2, r2, q2, gate=far(T, H, FAR, B, gate), yscales=s2, **kw)
    assert torch.equal(r2, r) and torch.equal(q2, q) and torch.equal(s2, s)


def test_linear_far_rows():
    """The largest strides, in place and laid out first, also of Y and of the scales."""
    M, N, K = 300, 48, 256
    g = torch.Generator("cuda").manual_seed(2)
    c, s = torch.empty((N, K), dtype=torch.uint8, device="cuda"), torch.empty((1, 2), device="cuda")
    sdg.spense_quantize_fp8b(torch.randn(N, K, device="cuda", generator=g), c, s, rows=128)
    layer = sdg.SpenseLinearFp8b(c, s)
    experts = sdg.SpenseExpertsFp8b(c[None], s[None])
    X = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    xq, xs = torch.empty((M, K), dtype=torch.uint8, device="cuda"), torch.empty((M, 2), device="cuda")
    sdg.spense_quantize_fp8b(X, xq, xs)
    pick = torch.randint(0, M, (M,), device="cuda", generator=g).int()
    off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    Y, Z = (torch.empty((M, N), device="cuda") for _ in range(2))
    layer(X, Y)
    experts(X, off, Z, rows=pick)
    for ld in ((1 << 22) - 8, (1 << 23) - 8):
        assert torch.equal(layer(far(M, K, ld, torch.bfloat16, X), far(M, N, 1 << 23, torch.float32)), Y), ld
    assert torch.equal(experts(far(M, K, (1 << 23) - 8, torch.bfloat16, X), off, torch.empty_like(Z), rows=pick), Z)
    layer.quantized(xq, xs, Y)
    experts.quantized(xq, xs, off, Z, rows=pick)
    for ld, lds in (((1 << 23) - 16, 2), (K, (1 << 21) - 1), (K, 1 << 21), ((1 << 23) - 1, (1 << 23) - 1)):
        q, t = far(M, K, ld, torch.uint8, xq), far(M, 2, lds, torch.float32, xs)
        assert torch.equal(layer.quantized(q, t, torch.empty_like(Y)), Y), (ld, lds)
        assert torch.equal(experts.quantized(q, t, off, torch.empty_like(Z), rows=pick), Z), (ld, lds)
    layer.close()
    experts.close()


def test_more_threads_than_a_launch():
    """2^33 values: rows past the first launch's come out as they do alone, and so do the products' activations."""
    M, K, N = 8200, 1 << 20, 16
    X = torch.empty((M, K), dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(3))
    at = [0, 8191, 8192, 8199]
    C, S = torch.empty((M, K), dtype=torch.uint8, device="cuda"), torch.empty((M, K // 128), device="cuda")
    sdg.spense_quantize_fp8b(X, C, S)
    c, s = torch.empty((4, K), dtype=torch.uint8, device="cuda"), torch.empty((4, K // 128), device="cuda")
    sdg.spense_quantize_fp8b(X[at], c, s)
    assert torch.equal(C[at], c) and torch.equal(S[at], s)

    wc, ws = torch.empty((N, K), dtype=torch.uint8, device="cuda"), torch.empty((1, K // 128), device="cuda")
    sdg.spense_quantize_fp8b(torch.randn(N, K, device="cuda").bfloat16(), wc, ws, rows=128)
    layer = sdg.SpenseLinearFp8b(wc, ws)
    x, W = oracle.fp8b_values_ref(c.cpu().numpy(), s.cpu().numpy()), oracle.fp8b_values_ref(wc.cpu().numpy(), ws.cpu().numpy(), 128)
    ref, B = oracle.product_ref(x, W)
    tol = product_tolerance(x, W, ref, B, K, True, torch.float32)
    Y = torch.empty((M, N), device="cuda")
    layer.w8a8(X, Y)
    assert_close(f64(Y[at]), ref, tol, "quantised in the call")
    Xc = torch.empty((M, K + 1), dtype=torch.uint8, device="cuda")[:, 1:]  # no row starts at 16 bytes
    Xc.copy_(C)
    layer.quantized(Xc, S, Y.zero_())
    assert_close(f64(Y[at]), ref, tol, "laid out")
    del Xc
    layer.close()

    back = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    sdg.spense_dequantize_fp8b(C, S, back)
    y = torch.empty((4, K), dtype=torch.bfloat16, device="cuda")
    sdg.spense_dequantize_fp8b(c, s, y)
    assert torch.equal(back[at], y)
    del back, C, S, X
    torch.cuda.empty_cache()
