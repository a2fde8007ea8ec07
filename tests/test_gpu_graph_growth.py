"""A graph captured at a small batch size and replayed after larger eager calls
on the same handle, which replace the workspaces that the graph holds: every
replay equals the eager call bit for bit."""

import numpy as np
import pytest
import torch

import oracle
import sparse_dense_gemm_amd as sdg
import synth
from synth import DT_BF16, DT_F32, DT_FP8

from spense_gpu_util import pack_dev, to_dev

pytestmark = pytest.mark.gpu

N, K, SMALL, LARGE = 96, 4096, 5, (70, 900)


def mx4(rows):
    c, s = oracle.mx4_quantize_ref(np.random.default_rng(1).standard_normal((rows, K)) * 0.02)
    return torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()


def sparse(dense_cols=None):
    W, s = synth.make_weight(N, K, DT_FP8, np.random.default_rng(2))
    kw = dict(dense_fraction=0.25) if dense_cols is None else dict(dense_cols=dense_cols)
    return pack_dev(to_dev(W, DT_FP8), DT_FP8, to_dev(s, DT_F32), **kw)


def make(kind):
    """The handle, and run(X, Y)."""
    if kind == "experts":
        codes, scales = mx4(3 * N)
        h = sdg.spense_pack_experts(codes.view(3, N, -1), sdg.DT_MX4, scales=scales.view(3, N, -1))

        def run(X, Y):
            sdg.spense_experts_linear(h, X, offsets[X.shape[0]], Y, adtype=sdg.DT_MX4)

        offsets = {M: torch.tensor([0, M // 3, M // 3, M], dtype=torch.int32, device="cuda") for M in (SMALL, *LARGE)}
        return h, run
    if kind in ("mx4", "w4a4"):
        h = sdg.spense_pack_mx4(*mx4(N))
        return h, lambda X, Y: (sdg.spense_linear_w4a4 if kind == "w4a4" else sdg.spense_linear)(h, X, Y)
    h = sparse(synth.random_dense_set(K, 1024, 3) if kind == "chosen" else None)
    return h, lambda X, Y: (sdg.spense_linear_w8a8 if kind == "w8a8" else sdg.spense_linear)(h, X, Y)


@pytest.mark.parametrize("kind", ["tail", "chosen", "w8a8", "mx4", "w4a4", "experts"])
def test_replays_after_larger_calls(kind):
    h, run = make(kind)
    try:
        X = to_dev(synth.make_x(LARGE[-1], K, DT_BF16, np.random.default_rng(4)), DT_BF16)
        eager = torch.empty((SMALL, N), device="cuda")
        Y = torch.empty_like(eager)
        run(X[:SMALL], eager)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(X[:SMALL], Y)
        torch.cuda.synchronize()
        for M in (SMALL, *LARGE):
            large = torch.empty((M, N), device="cuda")
            run(X[:M], large)                    # the last two replace the workspaces
            torch.cuda.synchronize()
            for _ in range(2):
                Y.fill_(float("nan"))
                graph.replay()
                torch.cuda.synchronize()
                assert torch.equal(Y, eager), (kind, M)
                again = torch.empty_like(large)
                run(X[:M], again)
                torch.cuda.synchronize()
                assert torch.equal(again, large), (kind, M)
    finally:
        sdg.spense_free(h)
