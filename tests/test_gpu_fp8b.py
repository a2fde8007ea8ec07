"""GPU parity of the fp8b format and linear layer (spense_quantize_fp8b,
spense_dequantize_fp8b, spense_pack_fp8b with spense_linear, spense_linear_w8a8
and spense_linear_fp8b) against the oracle.  Quantisation is compared bit for
bit, the products within the tolerances of fp8b_util.py."""

import numpy as np
import pytest
import torch

import oracle
import sparse_dense_gemm_amd as sdg

from fp8b_util import TYPES, acts, assert_close, bf16, dev, f64, product_tolerance, weights

pytestmark = pytest.mark.gpu


def quantize_dev(X, rows, pad=0):
    M, K = X.shape
    codes = torch.full((M, K + pad), 0x5A, dtype=torch.uint8, device="cuda")
    scales = torch.full((-(-M // rows), -(-K // 128) + pad), 7.0, device="cuda")
    sdg.spense_quantize_fp8b(X, codes, scales, rows=rows)
    torch.cuda.synchronize()
    assert (codes[:, K:] == 0x5A).all() and (scales[:, -(-K // 128):] == 7.0).all()  # what lies behind a row
    return codes[:, :K].cpu().numpy(), scales[:, :-(-K // 128)].cpu().numpy()


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 128), (3, 127), (5, 129), (128, 64), (129, 300), (300, 1000), (2, 5125)])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_quantize_bits(M, K, rows, t):
    rng = np.random.default_rng(M * 7 + K)
    x = (rng.standard_normal((M, K)) * 2.0 ** rng.integers(-30, 30, (M, 1))).astype(np.float32)
    X = dev(x) if t == "f32" else bf16(x)[0]
    want = oracle.fp8b_quantize_ref(X.float().cpu().numpy(), rows)
    for pad in (0, 3):
        got = quantize_dev(X, rows, pad)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]), (M, K, rows, t, pad)


def test_quantize_near_ties():
    """Quotients on, next to and near the borders between two codes, for scales of many mantissas and exponents."""
    v = oracle.e4m3_values()[:127]
    border = ((v[1:] + v[:-1]) / 2).astype(np.float32)
    rng = np.random.default_rng(3)
    rows = []
    for e in (-120, -91, -90, -89, -60, -1, 0, 40, 99, 100, 101, 110):
        for m in np.concatenate([[1.0, 1.5, 2 - 2.0 ** -23, 2 - 2.0 ** -22, 1 + 2.0 ** -23], 1 + rng.random(12)]):
            top = np.float32(m) * np.float32(2.0) ** e
            s = np.float32(top / np.float32(448))
            q = np.tile(border, 2)[:127] if s > 0 else np.zeros(127, np.float32)
            x = (q.astype(np.float64) * float(s if s > 0 else 1)).astype(np.float32)
            step = rng.integers(-2, 3, 127)
            x = np.minimum((x.view(np.int32) + step.astype(np.int32)).clip(0).view(np.float32), top)
            rows.append(np.concatenate([[top], x * np.where(rng.random(127) < 0.5, -1, 1)]).astype(np.float32))
    X = np.stack(rows)
    want = oracle.fp8b_quantize_ref(X)
    got = quantize_dev(dev(X), 1)
    assert np.array_equal(got[1], want[1])
    assert np.array_equal(got[0], want[0]), np.argwhere(got[0] != want[0])[:5].tolist()


def test_quantize_random_quotients():
    """The codes are those of the rounded quotient: 16 million quotients of numbers without structure."""
    g = torch.Generator("cuda").manual_seed(5)
    X = torch.randn((1 << 17, 128), device="cuda", generator=g)
    codes = torch.empty(X.shape, dtype=torch.uint8, device="cuda")
    scales = torch.empty((X.shape[0], 1), device="cuda")
    sdg.spense_quantize_fp8b(X, codes, scales)
    top = X.abs().amax(1, keepdim=True)
    s = top / torch.full_like(top, 448.0)
    assert torch.equal(scales, s)
    want = (X / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(codes, want)


@pytest.mark.parametrize("rows", [1, 128])
def test_quantize_special_values(rows):
    x = np.zeros((256, 384), dtype=np.float32)
    x[0, 0], x[0, 130], x[0, 260] = np.nan, np.inf, -np.inf
    x[130, 5], x[131, 6] = 3.4e38, -3.4e38      # the scale's quotient is large
    x[130, 133], x[130, 134] = 1e-45, -1e-45    # and 0
    x[140, 300:310], x[140, 310] = -0.0, 2.0 ** -126
    for X in (dev(x), dev(x).bfloat16()):
        want = oracle.fp8b_quantize_ref(X.float().cpu().numpy(), rows)
        got = quantize_dev(X, rows)
        assert np.array_equal(got[1], want[1], equal_nan=True) and np.array_equal(got[0], want[0])


@pytest.mark.parametrize("rows,M,K", [(1, 1, 1), (1, 5, 300), (128, 130, 257), (128, 256, 1024)])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_dequantize_bits(rows, M, K, t):
    rng = np.random.default_rng(K)
    c = rng.integers(0, 256, (M, K)).astype(np.uint8)
    s = (rng.random((-(-M // rows), -(-K // 128))) * 2.0 ** rng.integers(-40, 40)).astype(np.float32)
    want = oracle.fp8b_values_ref(c, s, rows).astype(np.float32)
    want = want if t == "f32" else dev(want).bfloat16().float().cpu().numpy()
    store = torch.full((M, K + 5), 9.0, dtype=TYPES[t], device="cuda")
    sdg.spense_dequantize_fp8b(dev(c), dev(s), store[:, :K], rows=rows)
    assert np.array_equal(store[:, :K].float().cpu().numpy(), want, equal_nan=True)
    assert (store[:, K:] == 9.0).all()


def run(layer, kind, X, xq, xs, Y):
    if kind == "bf16":
        layer(X, Y)
    elif kind == "w8a8":
        layer.w8a8(X, Y)
    else:
        layer.quantized(xq, xs, Y)


KINDS = ["bf16", "w8a8", "codes"]
SIZES = [(1, 1, 1), (1, 16, 128), (1, 257, 96), (2, 48, 130), (5, 100, 640), (16, 129, 129), (17, 272, 1000),
         (33, 33, 2049), (64, 300, 384), (70, 64, 8192), (130, 520, 400), (257, 1030, 272)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("kind", KINDS)
def test_linear(M, N, K, kind):
    c, s, W = weights(N, K, N + K)
    layer = sdg.SpenseLinearFp8b(dev(c), dev(s))
    assert layer.info["split"] == 5 and layer.info["weight_bytes"] == N * K + 4 * s.size
    X, x = bf16(acts(M, K, M))
    q, qs = oracle.fp8b_quantize_ref(x)
    if kind != "bf16":
        x = oracle.fp8b_values_ref(q, qs)
    ref, B = oracle.product_ref(x, W)
    xq, xs = dev(q), dev(qs)
    for yt in (torch.float32, torch.bfloat16):
        store = torch.full((M + 1, N + 3), 5.0, dtype=yt, device="cuda")
        Y = store[:M, :N]
        run(layer, kind, X, xq, xs, Y)
        tol = product_tolerance(x, W, ref, B, K, kind != "bf16", yt)
        assert_close(f64(Y), ref, tol, (M, N, K, kind, yt))
        assert (store[M] == 5.0).all() and (store[:, N:] == 5.0).all()  # rows and columns behind Y
        again = torch.empty((M, N), dtype=yt, device="cuda")
        run(layer, kind, X, xq, xs, again)
        assert torch.equal(again, Y)  # deterministic
    layer.close()


def test_in_call_quantisation_equals_given_codes():
    """spense_linear_w8a8 is the quantisation and the product: the same bits."""
    c, s, _ = weights(200, 700, 1)
    layer = sdg.SpenseLinearFp8b(dev(c), dev(s))
    X, _ = bf16(acts(40, 700, 2))
    xq, xs = torch.empty((40, 700), dtype=torch.uint8, device="cuda"), torch.empty((40, 6), device="cuda")
    sdg.spense_quantize_fp8b(X, xq, xs)
    for yt in (torch.float32, torch.bfloat16):
        Y, Z = (torch.empty((40, 200), dtype=yt, device="cuda") for _ in range(2))
        assert torch.equal(layer.w8a8(X, Y), layer.quantized(xq, xs, Z))


@pytest.mark.parametrize("kind", ["bf16", "codes"])
def test_alignment_and_strides(kind):
    """Rows that start anywhere, with any stride, scales with any stride: the same bits as the dense copy."""
    M, N, K = 37, 150, 384
    c, s, _ = weights(N, K, 5)
    layer = sdg.SpenseLinearFp8b(dev(c), dev(s))
    X, x = bf16(acts(M, K, 6))
    q, qs = oracle.fp8b_quantize_ref(x)
    Y = torch.empty((M, N), device="cuda")
    run(layer, kind, X, dev(q), dev(qs), Y)
    for first, more in ((1, 0), (0, 1), (3, 13), (16, 16), (8, 8)):
        flat = torch.full((M * (K + more) + 64,), 0x7F, dtype=torch.uint8, device="cuda")  # NaN codes between the rows
        xq = flat[first:first + M * (K + more)].view(M, K + more)[:, :K]
        xq.copy_(dev(q))
        xs = torch.full((M, 3 + more), float("nan"), device="cuda")[:, :3]
        xs.copy_(dev(qs))
        Xf = torch.full((M * (K + more) + 64,), float("nan"), dtype=torch.bfloat16, device="cuda")
        Xs = Xf[first:first + M * (K + more)].view(M, K + more)[:, :K]
        Xs.copy_(X)
        Z = torch.empty((M, N + 1), device="cuda")[:, :N]
        run(layer, kind, Xs, xq, xs, Z)
        assert torch.equal(Z, Y), (first, more)


@pytest.mark.parametrize("kind", KINDS)
def test_tail_columns_are_not_read(kind):
    """Columns from K on may hold NaN, in X, its scales and the weights' rows."""
    M, N = 20, 40
    for K in (64, 100, 144, 272, 304):
        c, s, W = weights(N, K, K)
        wide = torch.full((N, K + 48), 0x7F, dtype=torch.uint8, device="cuda")
        wide[:, :K] = dev(c)
        ws = torch.full((1, s.shape[1] + 2), float("nan"), device="cuda")
        ws[:, :s.shape[1]] = dev(s)
        layer = sdg.SpenseLinearFp8b(wide, ws, K=K)
        X, x = bf16(acts(M, K, K))
        q, qs = oracle.fp8b_quantize_ref(x)
        if kind != "bf16":
            x = oracle.fp8b_values_ref(q, qs)
        Xw = torch.full((M, K + 48), float("nan"), dtype=torch.bfloat16, device="cuda")
        Xw[:, :K] = X
        xw = torch.full((M, K + 48), 0x7F, dtype=torch.uint8, device="cuda")
        xw[:, :K] = dev(q)
        sw = torch.full((M, s.shape[1] + 2), float("nan"), device="cuda")
        sw[:, :s.shape[1]] = dev(qs)
        ref, B = oracle.product_ref(x, W)
        Y = torch.empty((M, N), device="cuda")
        run(layer, kind, Xw, xw, sw, Y)
        assert_close(f64(Y), ref, product_tolerance(x, W, ref, B, K, kind != "bf16", torch.float32), (kind, K))


def test_scales_of_any_size():
    """Zero, tiny and huge scales, and a NaN block in one row only."""
    M, N, K = 18, 200, 512
    c, s, _ = weights(N, K, 9)
    s = s * np.array([1e-30, 0.0, 1e25, 1.0], dtype=np.float32) * np.array([[1.0], [3.0]], dtype=np.float32)
    layer = sdg.SpenseLinearFp8b(dev(c), dev(s))
    W = oracle.fp8b_values_ref(c, s, 128)
    x = acts(M, K, 4)
    q, qs = oracle.fp8b_quantize_ref(x)
    qs[3, 2], qs[5, 0], qs[7] = 0.0, 1e10, 1e-20
    xv = oracle.fp8b_values_ref(q, qs)
    ref, B = oracle.product_ref(xv, W)
    for yt in (torch.float32, torch.bfloat16):
        Y = torch.empty((M, N), dtype=yt, device="cuda")
        layer.quantized(dev(q), dev(qs), Y)
        tol = product_tolerance(xv, W, ref, B, K, True, yt) + 2.0 ** -126 * K  # products of scales may be subnormal
        assert_close(f64(Y), ref, tol, yt)
        bad = qs.copy()
        bad[11, 1] = np.nan
        Z = torch.empty_like(Y)
        layer.quantized(dev(q), dev(bad), Z)
        rows = torch.arange(M, device="cuda") != 11
        assert torch.equal(Z[rows], Y[rows]) and Z[11].isnan().all()


def test_infinite_activations():
    """An infinity in bf16 activations reaches its row only; quantised, its row is NaN."""
    M, N, K = 5, 30, 256
    c, s, W = weights(N, K, 11)
    layer = sdg.SpenseLinearFp8b(dev(c), dev(s))
    X, x = bf16(acts(M, K, 12))
    Y, Z = torch.empty((M, N), device="cuda"), torch.empty((M, N), device="cuda")
    layer(X, Y)
    X[2, 200] = float("inf")
    layer(X, Z)
    rows = torch.tensor([0, 1, 3, 4], device="cuda")
    assert torch.equal(Y[rows], Z[rows])
    w = torch.from_numpy(W[:, 200]).cuda()
    assert torch.equal(Z[2].isinf(), w != 0) and torch.equal(Z[2] > 0, w > 0)
    layer.w8a8(X, Z)
    assert Z[2].isnan().all() and not Z[rows].isnan().any()


def test_refusals_on_a_handle():
    c, s, _ = weights(20, 200, 1)
    layer = sdg.SpenseLinearFp8b(dev(c), dev(s))
    lib, h = sdg._lib(), layer.handle
    X, Y = torch.zeros((4, 200), dtype=torch.bfloat16, device="cuda"), torch.zeros((4, 20), device="cuda")
    x, y = X.data_ptr(), Y.data_ptr()
    F32, BF16, FP8 = sdg.DT_F32, sdg.DT_BF16, sdg.DT_FP8
    assert lib.spense_linear(h, x, BF16, 4, 199, y, F32, 20, None) == sdg.SPENSE_EINVAL
    assert lib.spense_linear(h, x, F32, 4, 200, y, F32, 20, None) == sdg.SPENSE_EUNSUPPORTED
    assert lib.spense_linear(h, x, BF16, 4, 200, y, FP8, 20, None) == sdg.SPENSE_EUNSUPPORTED
    assert lib.spense_linear_splits(h, x, BF16, 4, 200, y, F32, 20, 2, None) == sdg.SPENSE_EUNSUPPORTED
    assert lib.spense_linear_noalloc(h, x, BF16, 4, 200, y, F32, 20, None) == sdg.SPENSE_EUNSUPPORTED
    assert lib.spense_linear_w8a8(h, x, 4, 200, y, F32, 20, 2, None) == sdg.SPENSE_EUNSUPPORTED
    assert lib.spense_linear_w4a4(h, x, 4, 200, y, F32, 20, None) == sdg.SPENSE_EUNSUPPORTED
    assert lib.spense_glu(h, x, 4, 200, x, 200, y, F32, 200, None) == sdg.SPENSE_EINVAL
    assert lib.spense_experts_linear(h, x, BF16, 4, 200, None, y, 4, y, F32, 20, None) == sdg.SPENSE_EINVAL
    assert lib.spense_experts_linear_fp8b(h, x, 200, y, 2, 4, None, y, 4, y, F32, 20, None) == sdg.SPENSE_EUNSUPPORTED
    assert lib.spense_export(h, None, None, None, None, None, None) == sdg.SPENSE_EINVAL
    for kw in (dict(ldc=199), dict(lds=1), dict(ldy=19), dict(M=0), dict(M=(1 << 24) + 1)):
        a = dict(ldc=200, lds=2, M=4, ldy=20)
        a.update(kw)
        assert lib.spense_linear_fp8b(h, x, a["ldc"], y, a["lds"], a["M"], y, F32, a["ldy"], None) == sdg.SPENSE_EINVAL
    assert lib.spense_linear_fp8b(h, x, 200, y, 2, 4, y, FP8, 20, None) == sdg.SPENSE_EUNSUPPORTED
    q, qs = torch.zeros((4, 200), dtype=torch.uint8, device="cuda"), torch.zeros((4, 2), device="cuda")
    for bad in (dict(codes=q[:, :199]), dict(scales=qs[:, :1]), dict(scales=qs[:3]), dict(Y=Y[:3]), dict(Y=Y[:, :19]),
                dict(codes=q.int()), dict(scales=qs.bfloat16())):
        a = dict(codes=q, scales=qs, Y=Y)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            layer.quantized(a["codes"], a["scales"], a["Y"])
    for X1, Y1 in ((X[:, :199], Y), (X, Y[:3]), (X, Y[:, :19])):
        for call in (layer, layer.w8a8):
            with pytest.raises(ValueError):
                call(X1, Y1)
    mx = sdg.SpenseLinearMx4(torch.zeros((20, 100), dtype=torch.uint8, device="cuda"),
                             torch.zeros((20, 7), dtype=torch.uint8, device="cuda"))
    assert lib.spense_linear_fp8b(mx.handle, x, 200, y, 2, 4, y, F32, 20, None) == sdg.SPENSE_EUNSUPPORTED


@pytest.mark.parametrize("kind", KINDS)
def test_every_configuration(kind, monkeypatch):
    """Each configuration of the kernel, with and without split sums."""
    M, N, K = 150, 600, 1500
    c, s, W = weights(N, K, 3)
    layer = sdg.SpenseLinearFp8b(dev(c), dev(s))
    X, x = bf16(acts(M, K, 4))
    q, qs = oracle.fp8b_quantize_ref(x)
    if kind != "bf16":
        x = oracle.fp8b_values_ref(q, qs)
    ref, B = oracle.product_ref(x, W)
    for yt in (torch.float32, torch.bfloat16):
        tol = product_tolerance(x, W, ref, B, K, kind != "bf16", yt)
        for config in range(4 if kind != "bf16" and yt == torch.float32 else 5):
            for splits in (1, 3, 6):
                monkeypatch.setenv("SPENSE_FP8B", f"{config},{splits}")
                Y = torch.full((M, N), float("nan"), dtype=yt, device="cuda")
                run(layer, kind, X, dev(q), dev(qs), Y)
                assert_close(f64(Y), ref, tol, (kind, yt, config, splits))


@pytest.mark.parametrize("kind", KINDS)
def test_prefill_size(kind):
    """Sampled rows and columns of a product at a prefill size."""
    M, N, K = 2047, 12288, 5120
    g = torch.Generator("cuda").manual_seed(7)
    Wd = 0.02 * torch.randn(N, K, device="cuda", generator=g)
    c, s = torch.empty((N, K), dtype=torch.uint8, device="cuda"), torch.empty((N // 128, K // 128), device="cuda")
    sdg.spense_quantize_fp8b(Wd, c, s, rows=128)
    layer = sdg.SpenseLinearFp8b(c, s)
    X = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    xq, xs = torch.empty((M, K), dtype=torch.uint8, device="cuda"), torch.empty((M, K // 128), device="cuda")
    sdg.spense_quantize_fp8b(X, xq, xs)
    m, n = np.r_[0:3, 126:130, 1000, 2040:2047], np.r_[0:3, 125:131, 6000:6017, 12280:12288]
    W = oracle.e4m3_values()[c[n].cpu().numpy()] * np.repeat(s.double().cpu().numpy()[n // 128], 128, 1)
    x = f64(X[m]) if kind == "bf16" else oracle.fp8b_values_ref(xq[m].cpu().numpy(), xs[m].cpu().numpy())
    ref, B = oracle.product_ref(x, W)
    for yt in (torch.float32, torch.bfloat16):
        Y = torch.empty((M, N), dtype=yt, device="cuda")
        run(layer, kind, X, xq, xs, Y)
        assert_close(f64(Y[m][:, n]), ref, product_tolerance(x, W, ref, B, K, kind != "bf16", yt), (kind, yt))
