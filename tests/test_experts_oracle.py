"""Pins of the oracle of the mx4 format, the experts' layers and the router:
hand-worked values, exhaustive properties and independent formulas."""

import numpy as np
import pytest

import oracle


def test_e2m1_rounding_by_hand():
    # numbers, midpoints (to the even code) and their neighbours
    cases = {0.0: 0, 0.25: 0, 0.2500001: 1, 0.5: 1, 0.75: 2, 0.7499: 1, 1.0: 2, 1.25: 2, 1.2501: 3, 1.5: 3, 1.75: 4,
             2.0: 4, 2.5: 4, 2.51: 5, 3.0: 5, 3.49: 5, 3.5: 6, 4.0: 6, 5.0: 6, 5.01: 7, 6.0: 7, 7.99: 7}
    got = oracle.nearest_e2m1(np.array(list(cases)))
    assert got.tolist() == list(cases.values())


def test_quantize_by_hand():
    x = np.zeros((5, 33))
    x[0, :4] = [6.0, -3.0, 0.5, -0.25]        # scale 1 (2^0: byte 127): codes 7, 8|5, 1, 8 (minus zero)
    x[1, 0], x[1, 31] = 1.0, -0.25            # largest 1 = 4 * 2^-2: byte 125, codes 6 and 8|2
    x[1, 32] = 2.0 ** -149                    # a lone subnormal: byte 0, far below half a step
    x[2, 3] = np.nan
    x[3, 0] = 7.9                             # saturates: byte 127, code 7
    x[4, 0] = 2.0 ** 127
    codes, scales = oracle.mx4_quantize_ref(x)
    assert scales.tolist() == [[127, 0], [125, 0], [255, 0], [127, 0], [252, 0]]
    assert codes[0, :2].tolist() == [7 | (13 << 4), 1 | (8 << 4)]
    assert codes[1, 0] == 6 and codes[1, 15] == (10 << 4) and codes[1, 16] == 0
    assert not codes[2].any()
    assert codes[3, 0] == 7 and codes[4, 0] == 6
    v = oracle.mx4_values_ref(codes, scales, 33)
    assert v[0, :4].tolist() == [6.0, -3.0, 0.5, 0.0] and np.isnan(v[2, :32]).all() and v[2, 32] == 0
    assert v[1, 0] == 1.0 and v[1, 31] == -0.25 and v[4, 0] == 2.0 ** 127


@pytest.mark.parametrize("K", [1, 31, 32, 33, 100])
def test_quantize_is_nearest_and_idempotent(K):
    rng = np.random.default_rng(K)
    x = (rng.standard_normal((9, K)) * 2.0 ** rng.integers(-20, 20, (9, 1))).astype(np.float32)
    codes, scales = oracle.mx4_quantize_ref(x)
    v = oracle.mx4_values_ref(codes, scales, K)
    step = np.ldexp(1.0, scales.astype(int) - 127).repeat(32, 1)[:, :K]
    # no e2m1 number is nearer, saturation aside
    grid = np.concatenate([oracle.experts.E2M1, -oracle.experts.E2M1])
    d = np.abs(x[..., None].astype(np.float64) - grid * step[..., None]).min(-1)
    assert np.array_equal(np.abs(x - v), d)
    # the largest magnitude of a block lands in [4, 8) steps
    pad = np.zeros((9, -(-K // 32) * 32))
    pad[:, :K] = np.abs(x) / step
    assert ((pad.reshape(9, -1, 32).max(-1) >= 4) & (pad.reshape(9, -1, 32).max(-1) < 8)).all()
    again = oracle.mx4_quantize_ref(v)
    assert np.array_equal(oracle.mx4_values_ref(*again, K), v)


def test_experts_linear_is_a_product_per_group():
    rng = np.random.default_rng(3)
    X, W = rng.standard_normal((7, 5)), rng.standard_normal((3, 4, 5))
    rows = np.array([6, 0, 2, 2, -1, 9, 3])
    Y, B = oracle.experts_linear_ref(X, W, [0, 2, 2, 6], rows)
    assert np.allclose(Y[:2], X[[6, 0]] @ W[0].T) and np.allclose(Y[2:4], X[[2, 2]] @ W[2].T)
    assert not Y[4:6].any() and np.isnan(Y[6]).all() and (B[:4] >= np.abs(Y[:4])).all()


def test_route_by_hand():
    inf, nan = np.inf, np.nan
    l = np.array([[1.0, 3.0, 3.0, 2.0], [nan, -inf, 0.0, -inf], [-inf, nan, -inf, -inf], [0.0, inf, 5.0, inf]])
    ids, w, off, rows, pos = oracle.route_ref(l, 2)
    assert ids.tolist() == [[1, 2], [2, -1], [-1, -1], [1, 3]]
    assert w.tolist() == [[0.5, 0.5], [1.0, 0.0], [0.0, 0.0], [0.5, 0.5]]
    assert off.tolist() == [0, 0, 2, 4, 5]
    assert rows.tolist() == [0, 3, 0, 1, 3, -1, -1, -1]
    assert pos.tolist() == [[0, 2], [3, -1], [-1, -1], [1, 4]]
    w2 = oracle.route_ref(l, 2, renormalize=False)[1]
    p = np.exp(l[0] - 3) / np.exp(l[0] - 3).sum()
    assert np.allclose(w2[0], [p[1], p[2]]) and w2[1, 0] == 1.0


def test_route_groups_are_a_permutation():
    l = np.random.default_rng(1).standard_normal((40, 9))
    ids, w, off, rows, pos = oracle.route_ref(l, 3)
    assert sorted(pos.ravel()) == list(range(120)) and np.allclose(w.sum(1), 1)
    for t in range(40):
        for j in range(3):
            assert rows[pos[t, j]] == t and off[ids[t, j]] <= pos[t, j] < off[ids[t, j] + 1]


def test_combine_skips_missing_rows():
    O = np.arange(6.0).reshape(3, 2)
    Y, B = oracle.combine_ref(O, np.array([[2, -1], [0, 7]]), np.array([[0.5, 9.0], [-2.0, 1.0]]))
    assert Y.tolist() == [[2.0, 2.5], [0.0, -2.0]] and B.tolist() == [[2.0, 2.5], [0.0, 2.0]]


def test_planted_mistakes_are_seen():
    """Variants of the definitions that a kernel could compute by mistake give other numbers on these inputs."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((4, 70)) * 3
    codes, scales = oracle.mx4_quantize_ref(x)
    v = oracle.mx4_values_ref(codes, scales, 70)
    swapped = (codes >> 4) | (codes << 4)                      # nibble order
    assert not np.array_equal(oracle.mx4_values_ref(swapped, scales, 70), v)
    assert not np.array_equal(oracle.mx4_values_ref(codes, scales + 1, 70), v)  # exponent bias
    # rounding towards zero instead of to the nearest
    down = np.searchsorted(oracle.experts.E2M1, np.abs(np.ldexp(x[:, :32], 127 - scales[:, :1].astype(int))), "right") - 1
    assert not np.array_equal(down, (codes[:, :16, None] >> np.array([0, 4]) & 7).reshape(4, 32))
