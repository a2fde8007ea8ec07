"""Pins of the oracle of the block-scaled 8-bit format and of the pass between
two blocks: closed forms, torch's e4m3 type, brute force."""

import numpy as np
import pytest
import torch

import oracle


def test_values_are_those_of_the_type():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    got = oracle.e4m3_values()
    assert np.array_equal(got[:127], want[:127]) and np.array_equal(got[128:255], want[128:255])
    assert np.isnan(got[127]) and np.isnan(got[255]) and got[0x7E] == 448 and got[1] == 2.0 ** -9


def test_nearest_by_brute_force():
    v = oracle.e4m3_values()[:127]
    between = (v[1:] + v[:-1]) / 2
    q = np.concatenate([v, between, np.nextafter(between, 0), np.nextafter(between, 500), [448, 460, 1e9]])
    for x in np.concatenate([q, -q]):
        d = np.abs(np.minimum(np.abs(x), 448.0) - v)
        near = np.flatnonzero(d == d.min())
        code = int(near[0]) if len(near) == 1 else int(near[near % 2 == 0][0])
        assert oracle.nearest_e4m3(np.array([x]))[0] == code | (128 if np.signbit(x) else 0), x
    assert oracle.nearest_e4m3(np.array([-0.0]))[0] == 128


@pytest.mark.parametrize("rows,M,K", [(1, 1, 1), (1, 3, 300), (128, 1, 128), (128, 130, 257)])
def test_quantize(rows, M, K):
    X = np.random.default_rng(M).standard_normal((M, K)).astype(np.float32)
    X[0, :2] = 0.0
    c, s = oracle.fp8b_quantize_ref(X, rows)
    v = oracle.fp8b_values_ref(c, s, rows)
    wide = np.repeat(np.repeat(s, rows, 0)[:M], 128, 1)[:, :K].astype(np.float64)
    # half a step: 2^-4 of a normal number, 2^-10 of the scale of a subnormal one; both quotients are rounded
    assert (np.abs(v - X) <= np.maximum(2.0 ** -4 * np.abs(X), 2.0 ** -10 * wide) * (1 + 2.0 ** -20)).all()
    for i in range(s.shape[0]):
        for b in range(s.shape[1]):
            x = X[i * rows:(i + 1) * rows, b * 128:(b + 1) * 128]
            assert s[i, b] == (np.float32(np.abs(x).max() / np.float32(448)) or 1.0)
            if np.abs(x).max() > 0:  # the largest magnitude takes the largest code
                assert (c[i * rows:(i + 1) * rows, b * 128:(b + 1) * 128] & 127).max() == 0x7E


def test_quantize_special_blocks():
    X = np.zeros((5, 128), dtype=np.float32)
    X[1, 3], X[2, 5], X[3, 7] = np.nan, -np.inf, 1e-45
    X[4] = 448.0
    c, s = oracle.fp8b_quantize_ref(X)
    assert s[0, 0] == 1 and not c[0].any()
    assert np.isnan(s[1, 0]) and np.isnan(s[2, 0]) and not c[1].any() and not c[2].any()
    assert s[3, 0] == 1 and not c[3].any()   # 1e-45 / 448 is 0 in 32 bits
    assert s[4, 0] == 1 and (c[4] == 0x7E).all()


def test_expert_scales_of_gate_and_up():
    """Gate and up count their blocks of rows from their own first row."""
    c = np.full((1, 400, 130), 0x38, dtype=np.uint8)  # ones
    s = np.arange(8, dtype=np.float32).reshape(1, 4, 2) + 1
    v = oracle.fp8b_expert_values_ref(c, s, True)[0]
    assert (v[:128, :128] == 1).all() and (v[128:200, :128] == 3).all() and (v[200:328, :128] == 5).all()
    assert (v[328:, 128:] == 8).all() and (v[199, 128:] == 4).all() and (v[200, 128:] == 6).all()
    assert (oracle.fp8b_expert_values_ref(c, s, False)[0][384:, 128:] == 8).all()


def test_dropped_bits_bound():
    x, w = np.ones((1, 16)), np.zeros((1, 16))
    w[0, 0], w[0, 9] = 4.0, 2.0
    assert oracle.dropped_bits_ref(x, w)[0, 0] == (4 + 2) * 2.0 ** -10


def test_block_norm_closed_form():
    O = np.array([[3.0, 4.0], [0.0, 0.0]])
    r, y, _ = oracle.block_norm_ref(O, eps=0.5, post=np.array([1.0, 2.0]), pre=np.array([2.0, 1.0]),
                                    gate=np.array([[0.5, 1.0]]), residual=np.array([[1.0, 0.0], [2.0, 0.0]]), scale=2.0)
    n = np.sqrt(12.5 + 0.5)
    assert np.allclose(r, [[2 + 1.5 / n, 8 / n], [4, 0]], rtol=1e-15)
    assert np.allclose(y[1], [8 / np.sqrt(8.5), 0], rtol=1e-15)
    m = np.sqrt((r[0] ** 2).mean() + 0.5)
    assert np.allclose(y[0], r[0] / m * [2, 1], rtol=1e-15)
    pos, weights = np.array([[1, 0], [5, -1]]), np.array([[0.5, 2.0], [1.0, 1.0]])
    r, _, o = oracle.block_norm_ref(O, eps=1.0, pos=pos, weights=weights)
    assert np.array_equal(o, [[6, 8], [0, 0]]) and np.array_equal(r, o)
