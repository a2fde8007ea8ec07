"""GPU parity of the experts' layers (spense_pack_experts,
spense_experts_linear) against the oracle, over group sizes that are empty,
single rows, tile edges and everything at once.

Tolerances as for the mx4 layer: the fp32 sum of exact products,
(K / 32 + 160) 2^-23 B.  With gate and up sums g, u off by e_g, e_u,
silu(g) u is off by at most 1.1 e_g (|u| + e_u) + |silu(g)| e_u (|silu'| <
1.1), the fast exponential by 2^-18 |silu(g) u|, and a bf16 output by 2^-8 of
itself.
"""

import numpy as np
import pytest
import torch

import oracle
import sparse_dense_gemm_amd as sdg

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def experts_case(E, N, K, wdtype, glu, seed):
    rng = np.random.default_rng(seed)
    w = (rng.standard_normal((E, N, K)) / np.sqrt(K)).astype(np.float32)
    if wdtype == sdg.DT_MX4:
        c, s = oracle.mx4_quantize_ref(w.reshape(E * N, K))
        W = oracle.mx4_values_ref(c, s, K).reshape(E, N, K)
        h = sdg.SpenseExperts(dev(c.reshape(E, N, -1)), sdg.DT_MX4, scales=dev(s.reshape(E, N, -1)), K=K, glu=glu)
    else:
        Wb = dev(w).bfloat16()
        W = Wb.float().cpu().numpy().astype(np.float64)
        h = sdg.SpenseExperts(Wb, sdg.DT_BF16, glu=glu)
    return h, W


def check(h, W, X, offsets, rows, R, glu, adtype=sdg.DT_BF16, yt=torch.float32, label=""):
    E, N, K = W.shape
    xr = X.float().cpu().numpy().astype(np.float64)
    if adtype == sdg.DT_MX4:
        xr = oracle.mx4_values_ref(*oracle.mx4_quantize_ref(xr), K)
    off = np.asarray(offsets, dtype=np.int32)
    ref, B = oracle.experts_linear_ref(xr, W, off, rows, R)
    eps = (K / 32 + 160) * 2.0 ** -23
    if glu:
        g, u = ref[:, :N // 2], ref[:, N // 2:]
        eg, eu = eps * B[:, :N // 2], eps * B[:, N // 2:]
        with np.errstate(over="ignore"):
            a = oracle.silu(g)
        ref = a * u
        tol = 1.1 * eg * (np.abs(u) + eu) + np.abs(a) * eu + 2.0 ** -18 * np.abs(ref)
    else:
        tol = eps * B
    if yt == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(ref)
    Y = torch.full((R, ref.shape[1]), 5.0, dtype=yt, device="cuda")
    h(X, dev(off), Y, rows=None if rows is None else dev(np.asarray(rows, dtype=np.int32)), adtype=adtype)
    y = Y.float().cpu().numpy().astype(np.float64)
    none = np.isnan(ref).all(1)
    assert (y[none] == 5.0).all(), (label, "rows of no expert were written")
    bad = ~(np.abs(y - ref) <= tol) & ~none[:, None]
    assert not bad.any(), (label, int(bad.sum()), np.argwhere(bad)[:4].tolist())


def offsets_of(sizes):
    return np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)


GROUPS = [
    [1], [0, 1], [1, 0, 0, 0], [0, 0, 0], [16, 17, 15, 1], [3, 0, 40, 0, 2], [0, 130, 0, 0, 300, 1],
    [64, 64], [5] * 9, [257, 0, 31], [1] * 70,
]
KINDS = [("bf16", "bf16"), ("mx4", "bf16"), ("mx4", "mx4")]


@pytest.mark.parametrize("w,a", KINDS, ids=lambda k: k)
@pytest.mark.parametrize("glu", [False, True], ids=["plain", "glu"])
@pytest.mark.parametrize("sizes", GROUPS, ids=lambda s: "x".join(map(str, s))[:20])
def test_groups(sizes, glu, w, a):
    E, (N, K) = len(sizes), (34, 136) if len(sizes) < 50 else (16, 64)
    rng = np.random.default_rng(sum(sizes) + E)
    h, W = experts_case(E, N, K, sdg.DT_MX4 if w == "mx4" else sdg.DT_BF16, glu, E)
    R = int(sum(sizes)) + 3                       # three rows of no expert
    M = max(1, R // 2)
    X = dev(rng.standard_normal((M, K)).astype(np.float32)).bfloat16()
    rows = rng.integers(0, M, R)
    if R > 4:
        rows[1], rows[2] = -1, M + 5              # outside X: zeros
    ad = sdg.DT_MX4 if a == "mx4" else sdg.DT_BF16
    check(h, W, X, offsets_of(sizes), rows, R, glu, ad, label=(sizes, w, a))
    Xg = dev(rng.standard_normal((R, K)).astype(np.float32)).bfloat16()
    check(h, W, Xg, offsets_of(sizes), None, R, glu, ad, torch.bfloat16, label=(sizes, w, a, "in place"))
    h.close()


@pytest.mark.parametrize("w,a", KINDS, ids=lambda k: k)
@pytest.mark.parametrize("N,K", [(2, 1), (18, 33), (100, 500), (256, 1030), (64, 2048), (500, 130)])
def test_sizes(N, K, w, a):
    sizes = [7, 0, 33, 1]
    rng = np.random.default_rng(N + K)
    for glu in (False, True):
        h, W = experts_case(4, N, K, sdg.DT_MX4 if w == "mx4" else sdg.DT_BF16, glu, N)
        X = dev(rng.standard_normal((20, K)).astype(np.float32)).bfloat16()
        rows = rng.integers(0, 20, 41)
        ad = sdg.DT_MX4 if a == "mx4" else sdg.DT_BF16
        for yt in (torch.float32, torch.bfloat16):
            check(h, W, X, offsets_of(sizes), rows, 41, glu, ad, yt, label=(N, K, glu))
        h.close()


def test_offsets_past_the_rows_are_cut():
    h, W = experts_case(3, 32, 64, sdg.DT_BF16, False, 1)
    X = dev(np.random.default_rng(1).standard_normal((10, 64)).astype(np.float32)).bfloat16()
    check(h, W, X, [0, 4, 9, 400], None, 10, False)


def test_strided_activations_and_outputs():
    h, W = experts_case(2, 20, 96, sdg.DT_MX4, False, 2)
    rng = np.random.default_rng(2)
    for start in (0, 1, 8):
        base = torch.full((9, 130), float("nan"), dtype=torch.bfloat16, device="cuda")
        base[:, start:start + 96] = dev(rng.standard_normal((9, 96)).astype(np.float32)).bfloat16()
        for ad in (sdg.DT_BF16, sdg.DT_MX4):
            check(h, W, base[:, start:start + 96], [0, 4, 9], None, 9, False, ad)


def test_graph_replays_follow_the_offsets():
    """The group sizes are read on the device: a captured call follows them from replay to replay."""
    E, N, K, R = 4, 64, 512, 48
    h, W = experts_case(E, N, K, sdg.DT_MX4, True, 3)
    rng = np.random.default_rng(3)
    X = dev(rng.standard_normal((R, K)).astype(np.float32)).bfloat16()
    rows = dev(rng.integers(0, R, R).astype(np.int32))
    off = dev(offsets_of([12, 12, 12, 12]))
    Y = torch.empty((R, N // 2), dtype=torch.float32, device="cuda")
    h(X, off, Y, rows=rows)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h(X, off, Y, rows=rows)
    for sizes in ([48, 0, 0, 0], [0, 1, 30, 17], [12, 12, 12, 12], [1, 2, 3, 42]):
        off.copy_(dev(offsets_of(sizes)))
        Y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        eager = torch.full_like(Y, float("nan"))
        h(X, off, eager, rows=rows)
        torch.cuda.synchronize()
        assert torch.equal(Y, eager) and not Y.isnan().any()


@pytest.mark.parametrize("w,a", KINDS, ids=lambda k: k)
@pytest.mark.parametrize("config", range(5))
def test_every_configuration_and_split(config, w, a, monkeypatch):
    """Each shape of the product kernel, with one and several splits of K, and other launch orders."""
    h, W = experts_case(3, 300, 1900, sdg.DT_MX4 if w == "mx4" else sdg.DT_BF16, False, 11)
    rng = np.random.default_rng(11)
    X = dev(rng.standard_normal((60, 1900)).astype(np.float32)).bfloat16()
    rows = rng.integers(0, 60, 290)
    ad = sdg.DT_MX4 if a == "mx4" else sdg.DT_BF16
    for plan in ("1", "2,1", "3,7", "4,3", "64"):
        monkeypatch.setenv("SPENSE_EXPERTS", f"{config},{plan}")
        check(h, W, X, [0, 17, 17, 287], rows, 290, False, ad, label=(config, plan))
    monkeypatch.setenv("SPENSE_EXPERTS", f"{config},2")
    outs = [torch.empty((290, 300), dtype=torch.float32, device="cuda") for _ in range(2)]
    for y in outs:
        h(X, dev(np.array([0, 17, 17, 290], dtype=np.int32)), y, rows=dev(rows.astype(np.int32)), adtype=ad)
    assert torch.equal(*outs)


def test_rows_past_31_bits_of_offset():
    """Activations of more than 2 GB: picked rows are gathered first, grouped ones read in place."""
    M, K, N = 300000, 4096, 32
    h, W = experts_case(2, N, K, sdg.DT_MX4, False, 12)
    X = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(12)
    pick = np.array([0, M - 1, 262143, 262144, 262145, 7])
    X[torch.from_numpy(pick).cuda()] = dev(rng.standard_normal((6, K)).astype(np.float32)).bfloat16()
    xs = X[torch.from_numpy(pick).cuda()].float().cpu().numpy().astype(np.float64)
    for ad in (sdg.DT_BF16, sdg.DT_MX4):
        xr = xs if ad == sdg.DT_BF16 else oracle.mx4_values_ref(*oracle.mx4_quantize_ref(xs), K)
        ref, B = oracle.experts_linear_ref(xr, W, [0, 2, 6])
        Y = torch.empty((6, N), dtype=torch.float32, device="cuda")
        h(X, dev(np.array([0, 2, 6], dtype=np.int32)), Y, rows=dev(pick.astype(np.int32)), adtype=ad)
        assert (np.abs(Y.cpu().numpy() - ref) <= (K / 32 + 160) * 2.0 ** -23 * B).all()
        # grouped already, the last rows beyond the offset
        Yb = torch.empty((M, N), dtype=torch.float32, device="cuda")
        h(X, dev(np.array([0, 5, M], dtype=np.int32)), Yb, adtype=ad)
        last, B = oracle.product_ref(xr[1:2], W[1])
        assert (np.abs(Yb[M - 1:].cpu().numpy() - last) <= (K / 32 + 160) * 2.0 ** -23 * B).all()


def test_one_eager_call_sizes_every_smaller_one():
    """Captures at smaller sizes than one eager call allocate nothing, whatever split count they take."""
    h, W = experts_case(4, 96, 4096, sdg.DT_MX4, False, 13)
    X = dev(np.random.default_rng(13).standard_normal((900, 4096)).astype(np.float32)).bfloat16()
    for ad in (sdg.DT_BF16, sdg.DT_MX4):
        Y = torch.empty((900, 96), dtype=torch.float32, device="cuda")
        off = dev(offsets_of([900, 0, 0, 0]))
        h(X[:20], off, Y[:20], adtype=ad)
        h(X, off, Y, adtype=ad)
        torch.cuda.synchronize()
        for R in (1, 17, 100, 333, 500, 777):
            out = torch.empty((R, 96), dtype=torch.float32, device="cuda")
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                h(X[:R], off, out, adtype=ad)
            for _ in range(2):
                out.fill_(float("nan"))
                graph.replay()
                torch.cuda.synchronize()
                h(X[:R], off, Y[:R], adtype=ad)
                torch.cuda.synchronize()
                assert torch.equal(out, Y[:R])


def test_refusals_on_a_handle():
    """Arguments that only a handle's sizes and types can refuse; nothing is written."""
    h, _ = experts_case(2, 32, 64, sdg.DT_BF16, True, 14)
    X = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    off = dev(np.array([0, 2, 4], dtype=np.int32))
    Y = torch.full((4, 16), 7.0, device="cuda")
    lib, ptr = sdg._lib(), [t.data_ptr() for t in (X, off, Y)]

    def call(adtype=sdg.DT_BF16, M=4, ldx=64, R=4, yt=sdg.DT_F32, ldy=16, rows=None, handle=h.handle):
        return lib.spense_experts_linear(handle, ptr[0], adtype, M, ldx, rows, ptr[1], R, ptr[2], yt, ldy, None)

    bad, unsupported = sdg.SPENSE_EINVAL, sdg.SPENSE_EUNSUPPORTED
    for kw, want in ((dict(M=0), bad), (dict(M=-1, R=0), bad), (dict(M=3), bad), (dict(M=0, rows=ptr[1]), bad),
                     (dict(R=-1), bad), (dict(ldx=63), bad), (dict(ldy=15), bad), (dict(adtype=9), bad),
                     (dict(yt=9), bad), (dict(adtype=sdg.DT_F32), unsupported), (dict(adtype=sdg.DT_MX4), unsupported),
                     (dict(yt=sdg.DT_FP8), unsupported), (dict(R=0, M=0), sdg.SPENSE_OK)):
        assert call(**kw) == want, kw
    # the other entry points do not take an experts' handle, nor this one theirs
    assert lib.spense_linear(h.handle, ptr[0], sdg.DT_BF16, 4, 64, ptr[2], sdg.DT_F32, 32, None) == bad
    assert lib.spense_linear_w4a4(h.handle, ptr[0], 4, 64, ptr[2], sdg.DT_F32, 32, None) == unsupported
    assert lib.spense_linear_w8a8(h.handle, ptr[0], 4, 64, ptr[2], sdg.DT_F32, 32, 0, None) == unsupported
    assert lib.spense_export(h.handle, None, None, None, None, None, None) == bad
    c, s = torch.zeros((32, 32), dtype=torch.uint8, device="cuda"), torch.zeros((32, 2), dtype=torch.uint8, device="cuda")
    layer = sdg.SpenseLinearMx4(c, s)
    assert call(handle=layer.handle) == bad
    assert lib.spense_linear_noalloc(layer.handle, ptr[0], sdg.DT_BF16, 4, 64, ptr[2], sdg.DT_F32, 32, None) == unsupported
    assert lib.spense_linear_splits(layer.handle, ptr[0], sdg.DT_BF16, 4, 64, ptr[2], sdg.DT_F32, 32, 2, None) == unsupported
    assert lib.spense_linear(layer.handle, ptr[0], sdg.DT_F32, 4, 64, ptr[2], sdg.DT_F32, 32, None) == unsupported
    assert lib.spense_linear(layer.handle, ptr[0], sdg.DT_BF16, 0, 64, ptr[2], sdg.DT_F32, 32, None) == bad
    torch.cuda.synchronize()
    assert (Y == 7.0).all()
    info = h.info
    assert (info["split"], info["N"], info["K"], info["N_s"], info["N_d"]) == (4, 32, 64, 2, 16)
