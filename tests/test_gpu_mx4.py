"""GPU parity of the mx4 format and the mx4 linear layer (spense_quantize_mx4,
spense_dequantize_mx4, spense_pack_mx4 with spense_linear and
spense_linear_w4a4) against the oracle.

Codes, exponent bytes and dequantised values are exact, so they are compared
bit for bit.  A product's only rounding is its fp32 sum: K / 32 matrix
instructions (each adding 32 or 128 products to an accumulator) and the split
sums, each off by at most 2^-23 of the sum of magnitudes B so far, so
  |Y - Yref| <= (K / 32 + 160) 2^-23 B,
the 160 covering the additions inside an instruction and the splits; a bf16
output adds 2^-8 |Yref|.
"""

import numpy as np
import pytest
import torch

import oracle
import sparse_dense_gemm_amd as sdg

pytestmark = pytest.mark.gpu


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def tolerance(K, B, Yref, bf16):
    return (K / 32 + 160) * 2.0 ** -23 * B + (2.0 ** -8 * np.abs(Yref) if bf16 else 0.0)


def quantize(X, ldc=0, lds=0):
    M, K = X.shape
    codes = torch.full((M, (K + 1) // 2 + ldc), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((M, -(-K // 32) + lds), 0xA5, dtype=torch.uint8, device="cuda")
    sdg.spense_quantize_mx4(X, codes, scales)
    torch.cuda.synchronize()
    return codes, scales


def random_x(M, K, rng, spread=20):
    x = rng.standard_normal((M, K)) * 2.0 ** rng.integers(-spread, spread, (M, 1))
    return x.astype(np.float32)


def hard_rows(K, rng):
    """Rows of midpoints, extremes, subnormals, zeros of both signs and non-finite values, in float32."""
    grid = np.array([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 7.0, 7.5])
    def row(lo, hi):
        s = 2.0 ** rng.integers(lo, hi + 1, -(-K // 32)).repeat(32)[:K]
        return (rng.choice(grid, K) * rng.choice([-1.0, 1.0], K) * s).astype(np.float32)

    out = [row(-10, 10), row(-126, -120), row(-149, -127), row(118, 124)]
    big = row(0, 0)
    big[::7] = np.finfo(np.float32).max
    out.append(big)
    out.append(np.zeros(K, np.float32) * -1.0)
    for bad in (np.nan, np.inf, -np.inf):
        r = row(-3, 3)
        r[K // 2] = bad
        out.append(r)
    tiny = np.zeros(K, np.float32)
    tiny[::3] = np.float32(1e-45)
    tiny[1::5] = -np.float32(3e-39)
    out.append(tiny)
    return np.stack(out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [1, 2, 7, 31, 32, 33, 64, 100, 257, 1000, 5120])
def test_quantize_bit_exact(K, dtype):
    rng = np.random.default_rng(K)
    x = np.concatenate([hard_rows(K, rng), random_x(13, K, rng)])
    X = dev(x)
    if dtype == "bf16":
        X = X.bfloat16()
        x = X.float().cpu().numpy()
    codes, scales = quantize(X)
    want_c, want_s = oracle.mx4_quantize_ref(x)
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    # back, exactly (a NaN block to NaN)
    v = oracle.mx4_values_ref(want_c, want_s, K)
    for yt in (torch.float32, torch.bfloat16):
        Y = torch.empty((x.shape[0], K), dtype=yt, device="cuda")
        sdg.spense_dequantize_mx4(codes, scales, Y)
        y = Y.float().cpu().numpy().astype(np.float64)
        assert np.array_equal(y, v, equal_nan=True)


def test_dequantize_every_code_and_exponent():
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))            # both halves take every code
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    want = oracle.mx4_values_ref(codes, scales, 512)
    for yt in (torch.float32, torch.bfloat16):
        Y = torch.empty((256, 512), dtype=yt, device="cuda")
        sdg.spense_dequantize_mx4(dev(codes), dev(scales), Y)
        y = Y.float().cpu().numpy().astype(np.float64)
        w = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)  # past the format's range
        assert np.array_equal(y, w, equal_nan=True)


def test_strides_and_offsets():
    """Rows of a larger matrix, starts off the 16-byte alignment, padding left alone."""
    rng = np.random.default_rng(9)
    for dtype in (torch.float32, torch.bfloat16):
        for K, start in ((64, 1), (96, 8), (33, 3)):
            base = dev(random_x(6, 150, rng)).to(dtype)
            X = base[:, start:start + K]
            codes, scales = quantize(X, ldc=3, lds=5)
            c, s = oracle.mx4_quantize_ref(X.float().cpu().numpy())
            codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
            assert np.array_equal(codes[:, :c.shape[1]], c) and (codes[:, c.shape[1]:] == 0xA5).all()
            assert np.array_equal(scales[:, :s.shape[1]], s) and (scales[:, s.shape[1]:] == 0xA5).all()
            Y = torch.full((6, 150), 7.0, dtype=dtype, device="cuda")
            sdg.spense_dequantize_mx4(dev(codes), dev(scales), Y[:, start:start + K])
            y = Y.float().cpu().numpy()
            assert np.array_equal(y[:, start:start + K], oracle.mx4_values_ref(c, s, K))
            assert (y[:, :start] == 7).all() and (y[:, start + K:] == 7).all()


def layer_case(N, K, seed):
    rng = np.random.default_rng(seed)
    codes, scales = oracle.mx4_quantize_ref(rng.standard_normal((N, K)) * 0.02)
    return sdg.SpenseLinearMx4(dev(codes), dev(scales), K=K), oracle.mx4_values_ref(codes, scales, K)


def check_linear(layer, W, x, yt=torch.float32, w4a4=False, X=None, label=""):
    M, K = x.shape
    X = dev(x).bfloat16() if X is None else X
    xr = X.float().cpu().numpy().astype(np.float64)
    if w4a4:
        xr = oracle.mx4_values_ref(*oracle.mx4_quantize_ref(xr), K)
    ref, B = oracle.product_ref(xr, W)
    Y = torch.full((M, W.shape[0]), float("nan"), dtype=yt, device="cuda")
    (layer.w4a4 if w4a4 else layer)(X, Y)
    y = Y.float().cpu().numpy().astype(np.float64)
    tol = tolerance(K, B, ref, yt == torch.bfloat16)
    bad = ~(np.abs(y - ref) <= tol)
    assert not bad.any(), (label, M, W.shape, int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(np.abs(y - ref)[bad].max()))
    return Y


@pytest.mark.parametrize("N,K", [(16, 128), (64, 512), (1, 1), (17, 33), (130, 1000), (48, 640), (200, 1600),
                                 (300, 4096), (33, 130)])
@pytest.mark.parametrize("w4a4", [False, True])
def test_linear_within_tolerance(N, K, w4a4):
    layer, W = layer_case(N, K, N + K)
    rng = np.random.default_rng(K)
    x = random_x(300, K, rng, 3)
    for M in (1, 2, 15, 16, 17, 33, 64, 65, 128, 129, 300):
        for yt in (torch.float32, torch.bfloat16):
            check_linear(layer, W, x[:M], yt, w4a4, label=(N, K, M, yt))
    assert layer.info["split"] == 3 and layer.info["N"] == N and layer.info["K"] == K
    layer.close()


@pytest.mark.parametrize("w4a4", [False, True])
def test_linear_reads_only_its_columns(w4a4):
    """NaN in the columns past K, in rows past M and around Y are neither read nor overwritten."""
    N, K = 50, 200
    layer, W = layer_case(N, K, 1)
    rng = np.random.default_rng(2)
    for start, ld in ((0, 208), (8, 216), (1, 209), (3, 203)):
        base = torch.full((40, ld), float("nan"), dtype=torch.bfloat16, device="cuda")
        x = random_x(20, K, rng, 2)
        base[:20, start:start + K] = dev(x).bfloat16()
        X = base[:20, start:start + K]
        xr = X.float().cpu().numpy().astype(np.float64)
        if w4a4:
            xr = oracle.mx4_values_ref(*oracle.mx4_quantize_ref(xr), K)
        ref, B = oracle.product_ref(xr, W)
        for ylead in (0, 1, 3):
            Yb = torch.full((22, N + 7), 3.0, dtype=torch.float32, device="cuda")
            Y = Yb[1:21, ylead:ylead + N]
            (layer.w4a4 if w4a4 else layer)(X, Y)
            y = Yb.cpu().numpy().astype(np.float64)
            assert (np.abs(y[1:21, ylead:ylead + N] - ref) <= tolerance(K, B, ref, False)).all(), (start, ylead)
            y[1:21, ylead:ylead + N] = 3.0
            assert (y == 3.0).all()


def test_nan_blocks_and_extreme_exponents():
    """A NaN block makes its output column NaN and no other; the smallest and largest exponents are taken as they are."""
    N, K = 40, 256
    rng = np.random.default_rng(4)
    codes, scales = oracle.mx4_quantize_ref(rng.standard_normal((N, K)))
    scales[3, 2] = 255
    scales[17, 5] = 255
    scales[20] = 0
    scales[21] = 190
    W = oracle.mx4_values_ref(codes, scales, K)
    layer = sdg.SpenseLinearMx4(dev(codes), dev(scales), K=K)
    x = rng.standard_normal((5, K)).astype(np.float32)
    X = dev(x).bfloat16()
    for w4a4 in (False, True):
        xr = X.float().cpu().numpy().astype(np.float64)
        if w4a4:
            xr = oracle.mx4_values_ref(*oracle.mx4_quantize_ref(xr), K)
        Y = torch.empty((5, N), dtype=torch.float32, device="cuda")
        (layer.w4a4 if w4a4 else layer)(X, Y)
        y = Y.cpu().numpy().astype(np.float64)
        assert np.isnan(y[:, [3, 17]]).all()
        ok = [n for n in range(N) if n not in (3, 17)]
        ref, B = oracle.product_ref(xr, W[ok])
        # sums below fp32's normal range may be flushed
        assert (np.abs(y[:, ok] - ref) <= tolerance(K, B, ref, False) + K * 2.0 ** -126).all()
    # a non-finite activation: its own row only
    X[2, 7] = float("inf")
    for w4a4 in (False, True):
        Y = torch.empty((5, N), dtype=torch.float32, device="cuda")
        (layer.w4a4 if w4a4 else layer)(X, Y)
        y = Y.cpu().numpy()
        assert np.isfinite(y[[0, 1, 3, 4]][:, ok]).all()
        assert not np.isfinite(y[2]).any() or not w4a4


def test_another_stream_and_graph():
    """On a stream of the caller's, and captured: replays equal the eager call bit for bit, also after a larger one."""
    N, K = 320, 2048
    layer, W = layer_case(N, K, 6)
    for w4a4 in (False, True):
        run = layer.w4a4 if w4a4 else layer
        X = dev(random_x(70, K, np.random.default_rng(7), 2)).bfloat16()
        Y = torch.empty((70, N), dtype=torch.float32, device="cuda")
        run(X, Y)                                             # sizes the workspaces of every smaller batch
        for M in (1, 40):
            eager = torch.empty((M, N), dtype=torch.float32, device="cuda")
            out = torch.empty_like(eager)
            run(X[:M], eager)
            torch.cuda.synchronize()
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                run(X[:M], out, stream=side)
            torch.cuda.synchronize()
            assert torch.equal(out, eager)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                run(X[:M], out)
            for _ in range(4):
                out.fill_(float("nan"))
                graph.replay()
                torch.cuda.synchronize()
                assert torch.equal(out, eager)
                run(X, Y)                                     # the program's own work between replays
                torch.cuda.synchronize()


def test_repeatable():
    layer, W = layer_case(160, 8192, 8)
    X = dev(random_x(24, 8192, np.random.default_rng(8), 2)).bfloat16()
    for run in (layer, layer.w4a4):
        a, b = (torch.empty((24, 160), dtype=torch.float32, device="cuda") for _ in range(2))
        run(X, a)
        run(X, b)
        assert torch.equal(a, b)
