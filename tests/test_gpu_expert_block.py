"""The expert block of examples/expert_block.py against the oracle, step by
step through its own intermediates, and as one HIP graph.

The router's choices are checked on the device's own logits; gate/up and down
on the weights its quantisation gives; the block's output is the oracle's
weighted sum of the oracle's down projections of the device's intermediate.
"""

import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle
import sparse_dense_gemm_amd as sdg

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("expert_block", os.path.join(ROOT, "examples", "expert_block.py"))
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def mx4(x):
    return oracle.mx4_values_ref(*oracle.mx4_quantize_ref(x), x.shape[1])


@pytest.mark.parametrize("adtype", [sdg.DT_BF16, sdg.DT_MX4], ids=["bf16", "mx4"])
@pytest.mark.parametrize("T", [1, 5, 70])
def test_block(T, adtype):
    E, H, I, k = 6, 192, 100, 2
    gate_up, down, router = example.make(E, H, I)
    block = example.ExpertBlock(gate_up, down, router, k, 70)
    X = torch.randn(T, H, device="cuda", generator=torch.Generator("cuda").manual_seed(T)).bfloat16()
    Y = torch.empty_like(X)
    block(X, Y, adtype)
    torch.cuda.synchronize()
    R = T * k
    logits = (X @ block.router.T).float().cpu().numpy()
    ids, w, off, rows, pos = oracle.route_ref(logits, k)
    assert np.array_equal(block.ids[:T].cpu().numpy(), ids) and np.array_equal(block.rows[:R].cpu().numpy(), rows)
    assert np.array_equal(block.offsets.cpu().numpy(), off) and np.array_equal(block.pos[:T].cpu().numpy(), pos)
    Wg = np.stack([mx4(f64(g)) for g in gate_up])
    Wd = np.stack([mx4(f64(d)) for d in down])
    x = f64(X) if adtype == sdg.DT_BF16 else mx4(f64(X))
    gu, B = oracle.experts_linear_ref(x, Wg, off, rows)
    g, u = gu[:, :I], gu[:, I:]
    eps = (H / 32 + 160) * 2.0 ** -23
    A = oracle.silu(g) * u
    tol = 1.1 * eps * B[:, :I] * (np.abs(u) + eps * B[:, I:]) + np.abs(oracle.silu(g)) * eps * B[:, I:]
    a_dev = f64(block.A[:R])
    assert (np.abs(a_dev - A) <= tol + (2.0 ** -8 + 2.0 ** -18) * np.abs(A)).all()
    a_in = a_dev if adtype == sdg.DT_BF16 else mx4(a_dev)
    O, B = oracle.experts_linear_ref(a_in, Wd, off)
    y, By = oracle.combine_ref(O, pos, w)
    _, Bo = oracle.combine_ref(B, pos, w)
    # the down sums' rounding, the weights' (E + 8 + logit range) and the sum's, then bf16
    tol = (I / 32 + 160) * 2.0 ** -23 * Bo + (E + 40) * 2.0 ** -23 * By + 2.0 ** -8 * np.abs(y)
    assert (np.abs(f64(Y) - y) <= tol).all()
    block.close()


def test_block_in_a_graph():
    """Captured with other tokens' routing from replay to replay."""
    E, H, I, k, T = 8, 256, 128, 2, 40
    block = example.ExpertBlock(*example.make(E, H, I), k, T)
    X = torch.randn(T, H, device="cuda").bfloat16()
    Y, eager = torch.empty_like(X), torch.empty_like(X)
    block(X, Y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(X, Y)
    for i in range(4):
        X.copy_(torch.randn(T, H, device="cuda").bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        got = Y.clone()
        block(X, eager)
        torch.cuda.synchronize()
        assert torch.equal(got, eager)
    block.close()
