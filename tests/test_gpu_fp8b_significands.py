"""Codes of fp8b for scales of chosen significands: all ones, where one Newton
step on a reciprocal that is a unit off can end on a tie, and its neighbours.
Compared with the oracle bit for bit.  (Values of bf16 have no such scales: 448
times a significand of all ones takes more than eight bits.)"""

import numpy as np
import pytest
import torch

import oracle
import sparse_dense_gemm_amd as sdg

from fp8b_util import dev

pytestmark = pytest.mark.gpu


def blocks():
    """Rows of 128: a top whose scale has the significand asked for, and values at the borders between codes, and next to
    them, of either sign; with the scales."""
    v = oracle.e4m3_values()[:127]
    border = (v[1:] + v[:-1]) / 2
    rng, rows = np.random.default_rng(1), []
    for e in range(-80, 101):
        for tail in (1, 2, 3, 0x7FFFFF):  # the scale (2 - tail 2^-23) 2^e
            s = (2 - tail * 2.0 ** -23) * 2.0 ** e
            top = np.float32(448 * s)
            assert np.float32(top / np.float32(448)) == np.float32(s)
            for step in (-1, 0, 1):
                x = (border * 2.0 ** (e + 1)).astype(np.float32)  # the quotients lie just above the borders
                x = (x.view(np.int32) + step).view(np.float32)
                x = np.minimum(x, top)
                rows.append(np.concatenate([[top], x * rng.choice([-1, 1], x.size), [0]]).astype(np.float32)[:128])
    return np.stack(rows)


@pytest.fixture(scope="module")
def given():
    x = blocks()
    c, s = oracle.fp8b_quantize_ref(x)
    assert (((s.view(np.uint32) & 0x7FFFFF) == 0x7FFFFF).mean() > 0.24)
    return x, c, s


def test_rows(given):
    x, want, scales = given
    c, s = torch.empty(x.shape, dtype=torch.uint8, device="cuda"), torch.empty((len(x), 1), device="cuda")
    sdg.spense_quantize_fp8b(dev(x), c, s)
    assert np.array_equal(s.cpu().numpy(), scales)
    assert np.array_equal(c.cpu().numpy(), want), np.argwhere(c.cpu().numpy() != want)[:4].tolist()


def test_blocks(given):
    """The same rows as blocks of 128 x 128: one of each in a block of copies."""
    x, want, scales = given
    at = np.arange(0, len(x), 37)
    X = np.repeat(x[at], 128, 0)
    c, s = torch.empty(X.shape, dtype=torch.uint8, device="cuda"), torch.empty((len(at), 1), device="cuda")
    sdg.spense_quantize_fp8b(dev(X), c, s, rows=128)
    assert np.array_equal(s.cpu().numpy(), scales[at]) and np.array_equal(c.cpu().numpy(), np.repeat(want[at], 128, 0))

