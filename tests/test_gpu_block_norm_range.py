"""The means of spense_block_norm at the end of fp32's range: a sum of squares
below 2^128 is finite and is divided by the columns like any other, one of 2^128
or more makes an infinite mean and the normalised row 0.

Sums in fp32 are off by at most n 2^-24 of themselves, n as in
test_gpu_block_norm.py (88 at 33001 columns, less below): 2^-17.  The rows' sums
are 2^-12 away from 2^128, so which side they fall on is not in doubt; the
tolerances are that file's."""

import numpy as np
import pytest
import torch

import sparse_dense_gemm_amd as sdg

from fp8b_util import TYPES, assert_close, dev, f64
from test_gpu_block_norm import reference, run

pytestmark = pytest.mark.gpu

TOP = 2.0 ** 128
SUMS = [1e38, 2.9e38, 3.0e38, 3.2e38, 3.35e38, TOP * (1 - 2.0 ** -12)]
OVER = [TOP * (1 + 2.0 ** -12), 1e39, 1e42]
LENGTHS = [1, 5, 8, 63, 256, 5120, 8199, 9000, 33001]


def rows(sums, H, seed, t="f32"):
    """A row for each sum of squares (before the values are rounded to the type)."""
    x = np.random.default_rng(seed).standard_normal((len(sums), H))
    x *= np.sqrt(np.asarray(sums) / (x * x).sum(1))[:, None]
    return dev(x.astype(np.float32)).to(TYPES[t])


def squares(O):
    return (f64(O) ** 2).sum(1)


@pytest.mark.parametrize("H", LENGTHS)
def test_large_finite_sums(H):
    """Both norms: of the block's output, and of the sum with the residual."""
    T = len(SUMS)
    O = rows(SUMS, H, H)
    assert (np.abs(squares(O) / SUMS - 1) < 2.0 ** -20).all()
    w = dev((1 + 0.2 * np.random.default_rng(1).standard_normal(H)).astype(np.float32))
    d = dict(O=O, post=w, gate=torch.full((H,), 0.5, device="cuda"), pre=w)
    r, y, dr, dy = reference(d, 0.75)
    R2, Y, _ = run(d, "f32", "f32", T, H)
    assert_close(f64(R2), r, dr, (H, "norm after the block"))
    assert_close(f64(Y), y, dy, (H, "and the next"))
    d = dict(O=O, pre=w)
    _, y, _, dy = reference(d, 0.75)
    for yt in ("f32", "bf16"):
        _, Y, _ = run(d, "f32", yt, T, H)
        assert_close(f64(Y), y, dy + (2.0 ** -8 if yt == "bf16" else 0.0) * np.abs(y), (H, yt, "norm before the next"))


@pytest.mark.parametrize("k", [0, 2])
def test_large_finite_sums_in_bf16(k):
    H, T = 712, len(SUMS) - 1
    O = rows(SUMS[:T] * max(k, 1), H, 3, "bf16")
    assert (squares(O) < TOP * (1 - 2.0 ** -12)).all() and (squares(O) > 0.99e38).all()
    d = dict(O=O, pre=torch.ones(H, device="cuda"))
    if k:  # the one row and nothing of the other
        d["pos"] = torch.stack([torch.arange(T), torch.arange(T) + T], 1).int().cuda()
        d["weights"] = torch.tensor([[1.0, 0.0]] * T, device="cuda")
    r, y, dr, dy = reference(d, 1.0)
    R2, Y, _ = run(d, "f32", "f32", T, H)
    assert_close(f64(R2), r, dr, "sum")
    assert_close(f64(Y), y, dy, "y")
    _, q, s = run(d, "f32", "fp8", T, H)
    c, t = torch.empty((T, H), dtype=torch.uint8, device="cuda"), torch.empty((T, 6), device="cuda")
    sdg.spense_quantize_fp8b(Y.contiguous(), c, t)
    assert torch.equal(q, c) and torch.equal(s, t)


@pytest.mark.parametrize("H", LENGTHS)
def test_sums_beyond(H):
    T = len(OVER)
    O = rows(OVER, H, H)
    w = torch.full((H,), 2.0, device="cuda")
    R2, Y, _ = run(dict(O=O, post=w, pre=w), "f32", "f32", T, H)
    assert (R2 == 0).all() and (Y == 0).all()
    R2, Y, _ = run(dict(O=O, pre=w), "f32", "f32", T, H)
    assert torch.equal(R2, O) and (Y == 0).all()
    _, q, s = run(dict(O=O), "f32", "fp8", T, H)
    assert (q & 127 == 0).all() and (s == 1).all()


@pytest.mark.parametrize("H", [7, 256, 5121])
def test_infinities_and_nan(H):
    """The infinite row: 0 but for its own place, which is a NaN; a NaN takes its row."""
    O = torch.ones((3, H), device="cuda")
    O[0, 3], O[1, 3] = float("inf"), float("nan")
    _, Y, _ = run(dict(O=O), "f32", "f32", 3, H)
    at = torch.arange(H, device="cuda") != 3
    assert (Y[0, at] == 0).all() and Y[0, 3].isnan() and Y[1].isnan().all() and (Y[2] - 1).abs().max() < 1e-5
