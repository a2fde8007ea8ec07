"""silu(gate) * up of a gate/up layer over the whole range of gate, with gate and
up sums that are exact (one product each).

With t = -g log2(e): its rounding and that of the constant move it by at most
|t| 2^-23, which moves 2^t by |g| 2^-23 of itself; the exponential and the
reciprocal instruction are good to 2^-23 each, the other four operations to
2^-24: (|g| + 4) 2^-23 in all.  exp(-g) passes the largest float at g = -88.73;
below, the result may be 0."""

import numpy as np
import pytest
import torch

import sparse_dense_gemm_amd as sdg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("up", [1.0, -2.0 ** 100, 2.0 ** -20])
def test_silu_over_the_range_of_gate(up):
    g = np.concatenate([np.linspace(-130, 130, 1041), np.linspace(-89, -87, 33), [0.0, -0.0, 2.0 ** -60, 3e38, 2.0 ** 20],
                        -np.array([2.0 ** -60, 0.5, 2.0 ** 20, 3e38])]).astype(np.float32)
    W = torch.zeros((1, 2 * g.size, 16), device="cuda")
    W[0, :g.size, 0] = torch.from_numpy(g).cuda()
    W[0, g.size:, 1] = up
    W = W.bfloat16()
    g = W[0, :g.size, 0].float().cpu().numpy().astype(np.float64)
    layer = sdg.SpenseExperts(W, glu=True)
    X = torch.zeros((1, 16), dtype=torch.bfloat16, device="cuda")
    X[0, :2] = 1.0
    Y = torch.empty((1, g.size), device="cuda")
    layer(X, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), Y)
    y = Y[0].cpu().numpy().astype(np.float64)
    with np.errstate(over="ignore", under="ignore"):
        want = g / (1 + np.exp(-g)) * up
        want = np.where(np.abs(want) < 2.0 ** 128, want, np.copysign(np.inf, want))
        tol = np.where(g < -88.7, 1.0, (np.abs(g) + 4) * 2.0 ** -23) * np.abs(want)
    # what is below the normal range after the factor `up`, or before it, may be flushed
    tol = np.where(np.isfinite(want), tol, 0) + 2.0 ** -126
    bad = ~((np.abs(y - want) <= tol) | (y == want))
    assert not bad.any(), [(float(a), float(b), float(c)) for a, b, c in zip(g[bad][:8], y[bad][:8], want[bad][:8])]
