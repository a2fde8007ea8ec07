"""GPU parity of the router and the weighted sum (spense_route,
spense_experts_combine) against the oracle.

Choices, groups and places are whole numbers and compared exactly.  A weight
is exp(l - max) over a sum of at most E such terms: the difference's rounding
(2^-24 of |l - max|, which shifts the exponential by that much), the
exponential (2 ulp), E additions and a division, so it is within
(|l - max| + E + 8) 2^-23 of itself.  The weighted sum takes k products and
additions: (k + 1) 2^-23 of the sum of magnitudes.
"""

import numpy as np
import pytest
import torch

import oracle
import sparse_dense_gemm_amd as sdg

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def route(L, k, renormalize=True):
    T, E = L.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, pos = torch.full((T, k), 77, **i32), torch.full((T, k), 77, **i32)
    weights = torch.full((T, k), 7.0, device="cuda")
    offsets, rows = torch.full((E + 1,), 77, **i32), torch.full((T * k,), 77, **i32)
    work = torch.full((max(1, sdg.spense_route_workspace(T, E, k)),), 0x5A, dtype=torch.uint8, device="cuda")
    sdg.spense_route(L, k, ids, weights, offsets, rows, pos, work, renormalize=renormalize)
    torch.cuda.synchronize()
    return ids, weights, offsets, rows, pos


def check(L, k, renormalize=True):
    l = L.float().cpu().numpy()
    got = [t.cpu().numpy() for t in route(L, k, renormalize)]
    want = oracle.route_ref(l, k, renormalize)
    for name, g, w in zip(("ids", "weights", "offsets", "rows", "pos"), got, want):
        if name != "weights":
            assert np.array_equal(g, w), (name, L.shape, k)
    with np.errstate(invalid="ignore"):
        top = np.where(np.isnan(l), -np.inf, l).max(1, keepdims=True)
        d = np.abs(np.take_along_axis(l, np.maximum(want[0], 0), 1) - top)
    d = np.where(np.isfinite(d), d, 0.0)
    tol = (d + L.shape[1] + 8) * 2.0 ** -23 * want[1] + 1e-37
    assert (np.abs(got[1] - want[1]) <= tol).all()


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 200])
@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (8, 2), (16, 1), (17, 4), (60, 6), (128, 8), (200, 8), (256, 3)])
def test_route(T, E, k):
    rng = np.random.default_rng(T * 1000 + E)
    L = dev(rng.standard_normal((T, E)).astype(np.float32) * 3)
    check(L, k)
    check(L.bfloat16(), k, renormalize=False)


@pytest.mark.parametrize("E,k", [(300, 5), (512, 10), (1024, 16), (1000, 1)])
def test_many_experts(E, k):
    L = dev(np.random.default_rng(E).standard_normal((70, E)).astype(np.float32))
    check(L, k)
    check(L, k, renormalize=False)


def test_ties_masks_and_extremes():
    rng = np.random.default_rng(0)
    T, E, k = 130, 24, 6
    l = rng.integers(-2, 3, (T, E)).astype(np.float32)          # many ties
    l[rng.random((T, E)) < 0.4] = -np.inf
    l[5] = -np.inf                                              # no expert left
    l[6] = np.nan
    l[7] = -np.inf
    l[7, 20] = -3.4e38                                          # one left, the lowest finite
    l[8, 3] = l[8, 9] = np.inf
    l[9, :] = np.inf
    l[10, ::2] = np.nan
    l[11, 0], l[11, 1] = -0.0, 0.0
    l[12] = np.finfo(np.float32).min                            # a mask of the lowest value masks nothing by itself
    l[13] = 0.0
    for renormalize in (True, False):
        check(dev(l), k, renormalize)
        check(dev(l).bfloat16(), k, renormalize)
    check(dev(l), E)


def test_all_tokens_to_one_expert_and_strides():
    base = torch.zeros((300, 40), device="cuda")
    base[:, 11] = 9.0
    check(base[:, 3:35], 1)
    check(base[:, 1:8], 7)


def test_blocks_beyond_the_first():
    """Token counts around the block sizes, with the counts of many blocks added up."""
    rng = np.random.default_rng(2)
    for T in (1025, 16385):
        l = rng.standard_normal((T, 8)).astype(np.float32)
        L = dev(l)
        ids, weights, offsets, rows, pos = (t.cpu().numpy() for t in route(L, 2))
        order = np.argsort(-l, axis=1, kind="stable")[:, :2]
        assert np.array_equal(ids, order)
        flat = order.ravel()
        at = np.argsort(flat, kind="stable")
        assert np.array_equal(rows, at // 2)
        assert np.array_equal(pos.ravel()[at], np.arange(2 * T))
        assert np.array_equal(offsets, np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=8))]))


def test_no_tokens():
    L = torch.empty((0, 5), device="cuda")
    _, _, offsets, _, _ = route(L, 2)
    assert not offsets.cpu().numpy().any()


def test_graph_and_stream():
    rng = np.random.default_rng(3)
    T, E, k = 150, 32, 4
    L = dev(rng.standard_normal((T, E)).astype(np.float32))
    outs = [torch.empty_like(t) for t in route(L, k)]
    work = torch.empty(max(1, sdg.spense_route_workspace(T, E, k)), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sdg.spense_route(L, k, *outs, work)
    for i in range(4):
        L.copy_(dev(rng.standard_normal((T, E)).astype(np.float32)))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, route(L, k)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("N", [1, 4, 7, 64, 1000])
@pytest.mark.parametrize("k", [1, 2, 9])
def test_combine(N, k):
    rng = np.random.default_rng(N + k)
    T, R = 37, 50
    pos = rng.integers(-1, R + 2, (T, k)).astype(np.int32)      # some missing, some outside
    pos[3] = -1
    w = rng.standard_normal((T, k)).astype(np.float32)
    for ot in (torch.float32, torch.bfloat16):
        O = torch.full((R, N + 3), float("nan"), dtype=ot, device="cuda")
        lead = N % 2
        O[:, lead:lead + N] = dev(rng.standard_normal((R, N)).astype(np.float32)).to(ot)
        Ov = O[:, lead:lead + N]
        ref, B = oracle.combine_ref(Ov.float().cpu().numpy().astype(np.float64), pos, w.astype(np.float64))
        for yt in (torch.float32, torch.bfloat16):
            Y = torch.full((T, N), 9.0, dtype=yt, device="cuda")
            sdg.spense_experts_combine(Ov, dev(pos), dev(w), Y)
            y = Y.float().cpu().numpy().astype(np.float64)
            tol = (k + 1) * 2.0 ** -23 * B + (2.0 ** -8 * np.abs(ref) if yt == torch.bfloat16 else 0)
            assert (np.abs(y - ref) <= tol).all()
            assert (y[3] == 0).all()


def test_combine_skips_missing_nan_rows():
    """A missing choice adds nothing, whatever lies where it would point."""
    O = torch.full((2, 8), float("nan"), device="cuda")
    O[1] = 2.0
    Y = torch.empty((1, 8), device="cuda")
    sdg.spense_experts_combine(O, dev(np.array([[1, -1]], dtype=np.int32)), dev(np.array([[0.5, 1.0]], dtype=np.float32)), Y)
    assert (Y == 1.0).all()
