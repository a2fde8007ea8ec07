"""GPU parity of the fp8b experts' layers (spense_pack_experts_fp8b with
spense_experts_linear and spense_experts_linear_fp8b) against the oracle, over
groups that are empty, single rows, tile edges and everything at once.

Tolerances of the sums: fp8b_util.py.  With gate and up sums g, u off by e_g, e_u,
silu(g) u is off by at most 1.1 e_g (|u| + e_u) + |silu(g)| e_u (|silu'| <
1.1), the fast exponential by 2^-18 |silu(g) u|, and a bf16 output by 2^-8 of
itself."""

import numpy as np
import pytest
import torch

import oracle
import sparse_dense_gemm_amd as sdg

from fp8b_util import acts, assert_close, bf16, dev, f64, product_tolerance

pytestmark = pytest.mark.gpu


def make(E, N, K, glu, seed):
    """Layer and float64 weights; gate and up are quantised on their own."""
    rng = np.random.default_rng(seed)
    w = (rng.standard_normal((E, N, K)) / np.sqrt(K)).astype(np.float32)
    codes, scales = [], []
    for e in range(E):
        parts = [w[e, :N // 2], w[e, N // 2:]] if glu else [w[e]]
        q = [oracle.fp8b_quantize_ref(p, 128) for p in parts]
        codes.append(np.concatenate([c for c, _ in q]))
        scales.append(np.concatenate([s for _, s in q]))
    c, s = np.stack(codes), np.stack(scales)
    return sdg.SpenseExpertsFp8b(dev(c), dev(s), glu=glu), oracle.fp8b_expert_values_ref(c, s, glu)


def reference(W, x, off, rows, R, glu, codes, yt):
    """Y and its tolerance [R, columns]; NaN on rows of no expert."""
    E, N, K = W.shape
    n = N // 2 if glu else N
    ref, tol = np.full((R, n), np.nan), np.full((R, n), np.nan)
    for e in range(E):
        at = np.arange(min(off[e], R), min(off[e + 1], R))
        if not len(at):
            continue
        src = at if rows is None else rows[at]
        xe = np.where(((src >= 0) & (src < len(x)))[:, None], x[np.clip(src, 0, len(x) - 1)], 0.0)
        y, B = oracle.product_ref(xe, W[e])
        if not glu:
            ref[at], tol[at] = y, product_tolerance(xe, W[e], y, B, K, codes, yt)
            continue
        # the sums themselves are not rounded to the output's type, but the codes' instruction goes with it
        t = product_tolerance(xe, W[e], 0 * y, B, K, codes, yt)
        g, u, eg, eu = y[:, :n], y[:, n:], t[:, :n], t[:, n:]
        a = oracle.silu(g)
        ref[at] = a * u
        tol[at] = 1.1 * eg * (np.abs(u) + eu) + np.abs(a) * eu + 2.0 ** -18 * np.abs(a * u)
        if yt == torch.bfloat16:
            tol[at] += 2.0 ** -8 * np.abs(a * u)
    return ref, tol


def check(h, W, X, off, rows, R, glu, kind, yt, label):
    K = W.shape[2]
    x = f64(X)
    q, qs = oracle.fp8b_quantize_ref(x)
    if kind != "bf16":
        x = oracle.fp8b_values_ref(q, qs)
    off = np.asarray(off, dtype=np.int32)
    rows = None if rows is None else np.asarray(rows, dtype=np.int32)
    ref, tol = reference(W, x, off, rows, R, glu, kind != "bf16", yt)
    Y = torch.full((R, ref.shape[1]), 5.0, dtype=yt, device="cuda")
    rd = None if rows is None else dev(rows)
    if kind == "codes":
        h.quantized(dev(q), dev(qs), dev(off), Y, rows=rd)
    else:
        h(X, dev(off), Y, rows=rd, adtype=sdg.DT_FP8 if kind == "call" else sdg.DT_BF16)
    y = f64(Y)
    none = np.isnan(ref).all(1)
    assert (y[none] == 5.0).all(), (label, "rows of no expert were written")
    assert_close(y[~none], ref[~none], tol[~none], label)


def offsets_of(sizes):
    return np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)


GROUPS = [[1], [0, 1], [1, 0, 0, 0], [0, 0, 0], [16, 17, 15, 1], [3, 0, 40, 0, 2], [0, 130, 0, 0, 300, 1],
          [64, 64], [5] * 9, [257, 0, 31], [1] * 70]


@pytest.mark.parametrize("kind", ["bf16", "call", "codes"])
@pytest.mark.parametrize("glu", [False, True], ids=["plain", "glu"])
@pytest.mark.parametrize("sizes", GROUPS, ids=lambda s: "-".join(map(str, s))[:20])
def test_groups(sizes, glu, kind):
    E, N, K = len(sizes), 76, 200
    h, W = make(E, N, K, glu, 1)
    R = int(sum(sizes))
    X, _ = bf16(acts(max(R, 1), K, R))
    for yt in (torch.float32, torch.bfloat16):
        check(h, W, X, offsets_of(sizes), None, R, glu, kind, yt, (sizes, glu, kind, yt))


@pytest.mark.parametrize("kind", ["bf16", "call", "codes"])
@pytest.mark.parametrize("N,K", [(2, 1), (400, 130), (516, 300), (1030, 512), (34, 1700)])
def test_shapes_with_picked_rows(N, K, kind):
    """Gate and up blocks that do not end on a row tile; rows picked, repeated and out of range."""
    E, M = 4, 45
    h, W = make(E, N, K, True, N)
    rng = np.random.default_rng(K)
    R = 150
    rows = rng.integers(-2, M + 3, R)
    off = [0, 20, 20, 149, R - 3]  # the last rows belong to none
    X, _ = bf16(acts(M, K, 3))
    for yt in (torch.float32, torch.bfloat16):
        check(h, W, X, off, rows, R, True, kind, yt, (N, K, kind, yt))


@pytest.mark.parametrize("kind", ["bf16", "codes"])
def test_offsets_of_any_kind(kind):
    """Offsets past R count as R; fewer rows picked than X has."""
    h, W = make(3, 40, 144, False, 5)
    X, _ = bf16(acts(400, 144, 6))
    rows = np.arange(30)[::-1] * 13
    check(h, W, X, [0, 7, 1000, 2000], rows, 30, False, kind, torch.float32, kind)
    check(h, W, X, [0, 0, 0, 0], rows, 30, False, kind, torch.float32, kind)


@pytest.mark.parametrize("kind", ["bf16", "codes"])
def test_every_configuration(kind, monkeypatch):
    h, W = make(5, 520, 1100, True, 8)
    off = offsets_of([90, 0, 33, 260, 1])
    X, _ = bf16(acts(100, 1100, 9))
    rows = np.random.default_rng(1).integers(0, 100, 384)
    for yt in (torch.float32, torch.bfloat16):
        for config in range(4 if kind != "bf16" and yt == torch.float32 else 5):
            for splits in (1, 4):
                monkeypatch.setenv("SPENSE_FP8B", f"{config},{splits}")
                check(h, W, X, off, rows, 384, True, kind, yt, (kind, yt, config, splits))


def test_no_rows_and_refusals():
    h, W = make(3, 40, 144, False, 5)
    lib, P = sdg._lib(), 1 << 20
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    Y = torch.empty((0, 40), device="cuda")
    h(torch.empty((0, 144), dtype=torch.bfloat16, device="cuda"), off, Y)
    h.quantized(torch.empty((0, 144), dtype=torch.uint8, device="cuda"), torch.empty((0, 2), device="cuda"), off, Y)
    F32, BF16, FP8, MX4 = sdg.DT_F32, sdg.DT_BF16, sdg.DT_FP8, sdg.DT_MX4

    def run(adtype=BF16, M=4, ldx=144, R=4, ldy=40, yt=F32, offsets=P):
        return lib.spense_experts_linear(h.handle, P, adtype, M, ldx, None, offsets, R, P, yt, ldy, None)

    for kw, want in ((dict(adtype=MX4), -2), (dict(adtype=F32), -2), (dict(adtype=9), -1), (dict(M=3), -1),
                     (dict(ldx=143), -1), (dict(ldy=39), -1), (dict(yt=FP8), -2), (dict(offsets=None), -1)):
        assert run(**kw) == want, kw

    def runq(codes=P, ldc=144, scales=P, lds=2, M=4, R=4, ldy=40, yt=F32, offsets=P):
        return lib.spense_experts_linear_fp8b(h.handle, codes, ldc, scales, lds, M, None, offsets, R, P, yt, ldy, None)

    for kw, want in ((dict(codes=None), -1), (dict(scales=None), -1), (dict(offsets=None), -1), (dict(ldc=143), -1),
                     (dict(lds=1), -1), (dict(M=3), -1), (dict(R=-1), -1), (dict(ldy=39), -1), (dict(yt=FP8), -2),
                     (dict(ldc=1 << 23), -2), (dict(R=0, codes=None, scales=None, M=0), 0)):
        assert runq(**kw) == want, kw
    assert lib.spense_linear(h.handle, P, BF16, 4, 144, P, F32, 40, None) == -1
    assert lib.spense_linear_fp8b(h.handle, P, 144, P, 2, 4, P, F32, 40, None) == -2
    q, s, Y = torch.zeros((4, 144), dtype=torch.uint8, device="cuda"), torch.zeros((4, 2), device="cuda"), torch.zeros((4, 40), device="cuda")
    for kw in (dict(off=off[:3]), dict(off=off.long()), dict(Y=Y[:, :39]), dict(rows=off[:3]), dict(rows=off.float()),
               dict(q=q[:, :143]), dict(s=s[:3])):
        a = dict(q=q, s=s, off=off, Y=Y, rows=None)
        a.update(kw)
        with pytest.raises((ValueError, TypeError)):
            h.quantized(a["q"], a["s"], a["off"], a["Y"], rows=a["rows"])
    experts = sdg.SpenseExperts(torch.zeros((2, 16, 64), dtype=torch.bfloat16, device="cuda"))
    assert lib.spense_experts_linear(experts.handle, P, FP8, 4, 64, None, P, 4, P, F32, 16, None) == -2
    assert lib.spense_experts_linear_fp8b(experts.handle, P, 64, P, 1, 4, None, P, 4, P, F32, 16, None) == -2


@pytest.mark.parametrize("kind", ["bf16", "codes"])
def test_prefill_size(kind):
    """Sampled rows of 16 experts at a prefill size, skewed groups."""
    E, I, K, T, k = 16, 1600, 5120, 4093, 2
    g = torch.Generator("cuda").manual_seed(3)
    c = torch.empty((E, 2 * I, K), dtype=torch.uint8, device="cuda")
    s = torch.empty((E, 26, 40), device="cuda")
    for e in range(E):
        for p in range(2):
            sdg.spense_quantize_fp8b(0.02 * torch.randn(I, K, device="cuda", generator=g), c[e, p * I:(p + 1) * I],
                                     s[e, 13 * p:13 * p + 13], rows=128)
    h = sdg.SpenseExpertsFp8b(c, s, glu=True)
    X = torch.randn(T, K, device="cuda", generator=g).bfloat16()
    logits = torch.randn(T, E, device="cuda", generator=g) + 0.8 * torch.randn(E, device="cuda", generator=g)
    flat = torch.topk(logits, k, 1)[1].flatten()
    order = torch.sort(flat, stable=True)[1]
    rows = (order // k).int()
    off = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), torch.bincount(flat, minlength=E).cumsum(0)]).int()
    xq, xs = torch.empty((T, K), dtype=torch.uint8, device="cuda"), torch.empty((T, 40), device="cuda")
    sdg.spense_quantize_fp8b(X, xq, xs)
    Y = torch.empty((T * k, I), dtype=torch.bfloat16, device="cuda")
    if kind == "bf16":
        h(X, off, Y, rows=rows)
    else:
        h.quantized(xq, xs, off, Y, rows=rows)
    o = off.cpu().numpy()
    n = np.r_[0:3, 127:130, 1590:1600]
    for e in (0, 7, 15):
        r = np.unique(np.clip(np.r_[o[e]:o[e] + 2, o[e] + 127:o[e] + 130, o[e + 1] - 2:o[e + 1]], o[e], o[e + 1] - 1))
        src = rows[r].long()
        x = f64(X[src]) if kind == "bf16" else oracle.fp8b_values_ref(xq[src].cpu().numpy(), xs[src].cpu().numpy())
        W = np.concatenate([oracle.e4m3_values()[c[e, p * I + n].cpu().numpy()]
                            * np.repeat(s[e, 13 * p + n // 128].double().cpu().numpy(), 128, 1) for p in range(2)])
        ref, tol = reference(W[None], x, [0, len(r)], None, len(r), True, kind != "bf16", torch.bfloat16)
        assert_close(f64(Y[r][:, n]), ref, tol, (kind, e))
