"""GPU parity of the products with mx4 and expert weights at prefill sizes (the
36B-class layer, and the 32B-class FFN cut into 16 experts, with ragged rows):
launches of many row groups and m-groups over all XCDs.  Sampled rows and
columns are compared with the oracle, the edges of the tiles among them; every
other output has to be finite.  Tolerances as in test_gpu_mx4 and
test_gpu_experts."""

import numpy as np
import pytest
import torch

import oracle
import sparse_dense_gemm_amd as sdg
from test_gpu_experts import KINDS
from test_gpu_mx4 import tolerance

pytestmark = pytest.mark.gpu


def random_mx4(shape, K, seed):
    """Codes and exponent bytes of weights of about 0.02, made on the device."""
    g = torch.Generator("cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (*shape, (K + 1) // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(119, 123, (*shape, -(-K // 32)), dtype=torch.uint8, device="cuda", generator=g)
    return codes, scales


def values(codes, scales, K):
    return oracle.mx4_values_ref(codes.cpu().numpy(), scales.cpu().numpy(), K)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def activations(M, K, seed):
    return torch.randn(M, K, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).bfloat16()


def sampled(n, edge, count, seed):
    """Indices below n: both ends, around multiples of `edge`, and random ones."""
    rng = np.random.default_rng(seed)
    near = (np.arange(0, n, edge)[:, None] + np.array([-1, 0, 1])).ravel()
    near = rng.permutation(near)[:count // 2]
    i = np.concatenate([[0, n - 1], near, rng.integers(0, n, count // 2)])
    return np.unique(i[(i >= 0) & (i < n)])


@pytest.mark.parametrize("a4", [False, True], ids=["bf16", "mx4"])
@pytest.mark.parametrize("M,N,K", [(2047, 12288, 5120), (257, 5121, 27648), (2000, 12290, 1030)])
def test_linear(M, N, K, a4):
    codes, scales = random_mx4((N,), K, N)
    layer = sdg.SpenseLinearMx4(codes, scales, K=K)
    X = activations(M, K, M)
    Y = torch.full((M, N), float("nan"), device="cuda")
    (layer.w4a4 if a4 else layer)(X, Y)
    assert Y.isfinite().all()
    r, c = sampled(M, 16, 40, 1), sampled(N, 256, 300, 2)
    rt, ct = torch.from_numpy(r).cuda(), torch.from_numpy(c).cuda()
    x = f64(X[rt])
    if a4:
        x = oracle.mx4_values_ref(*oracle.mx4_quantize_ref(x), K)
    ref, B = oracle.product_ref(x, values(codes[ct], scales[ct], K))
    y = f64(Y[rt][:, ct])
    assert (np.abs(y - ref) <= tolerance(K, B, ref, False)).all()
    Yb = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    (layer.w4a4 if a4 else layer)(X, Yb)
    assert torch.equal(Yb, Y.bfloat16())          # the same sums, rounded
    layer.close()


@pytest.mark.parametrize("w,a", KINDS, ids=lambda k: k)
@pytest.mark.parametrize("glu", [True, False], ids=["gate/up", "down"])
def test_experts(glu, w, a):
    E, H, I, T, k = 16, 5120, 1600, 4093, 2
    N, K = (2 * I, H) if glu else (H, I)
    R = T * k
    if w == "mx4":
        codes, scales = random_mx4((E, N), K, K)
        layer = sdg.SpenseExperts(codes, sdg.DT_MX4, scales=scales, K=K, glu=glu)
    else:
        g = torch.Generator("cuda").manual_seed(K)
        W = torch.stack([torch.randn(N, K, device="cuda", generator=g).mul_(0.02).bfloat16() for _ in range(E)])
        layer = sdg.SpenseExperts(W, glu=glu)
    rng = np.random.default_rng(K)
    sizes = rng.multinomial(R - 40, rng.dirichlet(np.ones(E - 1)))
    sizes = np.concatenate([sizes[:5], [0], sizes[5:]])       # one expert without rows, 40 rows of no expert
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    X = activations(T if glu else R, K, T)
    rows = rng.integers(0, T, R).astype(np.int32) if glu else None
    ad = sdg.DT_MX4 if a == "mx4" else sdg.DT_BF16
    Y = torch.full((R, I if glu else N), float("nan"), device="cuda")
    layer(X, torch.from_numpy(off).cuda(), Y, rows=None if rows is None else torch.from_numpy(rows).cuda(), adtype=ad)
    have = int(off[-1])
    assert Y[:have].isfinite().all() and Y[have:].isnan().all()
    cols = sampled(Y.shape[1], 128, 300, 3)
    pick = np.concatenate([cols, I + cols]) if glu else cols
    eps = (K / 32 + 160) * 2.0 ** -23
    for e in range(E):
        if not sizes[e]:
            continue
        r = off[e] + sampled(int(sizes[e]), 16, 12, e)
        src = torch.from_numpy(rows[r] if glu else r).cuda().long()
        x = f64(X[src])
        if ad == sdg.DT_MX4:
            x = oracle.mx4_values_ref(*oracle.mx4_quantize_ref(x), K)
        pt = torch.from_numpy(pick).cuda()
        We = values(codes[e][pt], scales[e][pt], K) if w == "mx4" else f64(W[e][pt])
        ref, B = oracle.product_ref(x, We)
        if glu:
            n = cols.size
            g, u, eg, eu = ref[:, :n], ref[:, n:], eps * B[:, :n], eps * B[:, n:]
            s = oracle.silu(g)
            ref, tol = s * u, 1.1 * eg * (np.abs(u) + eu) + np.abs(s) * eu + 2.0 ** -18 * np.abs(s * u)
        else:
            tol = eps * B
        y = f64(Y[torch.from_numpy(r).cuda().long()][:, torch.from_numpy(cols).cuda()])
        assert (np.abs(y - ref) <= tol).all(), e
    layer.close()
