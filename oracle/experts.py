"""Oracle of the microscaled 4-bit (mx4) format, the products with it, the
experts' layers and the router: plain NumPy in float64, from the definitions.

An mx4 value is an e2m1 number (sign; exponent and fraction as in
``E2M1``) times a power of two that 32 consecutive columns of a row share.
Every e2m1 number times a power of two is a float64, and so is every product
of two of them, so quantisation and dequantisation are exact here and a
product's only rounding is float64's sum.
"""

from __future__ import annotations

import numpy as np

BLOCK = 32
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx4_quantize_ref(X):
    """Codes [M, ceil(K/2)] and exponent bytes [M, ceil(K/32)] of float X [M, K]."""
    X = np.asarray(X, dtype=np.float64)
    M, K = X.shape
    codes = np.zeros((M, (K + 1) // 2), dtype=np.uint8)
    scales = np.zeros((M, -(-K // BLOCK)), dtype=np.uint8)
    for b in range(scales.shape[1]):
        x = X[:, b * BLOCK:(b + 1) * BLOCK]
        finite = np.isfinite(x).all(1)
        x = np.where(finite[:, None], x, 0.0)
        top = np.abs(x).max(1)
        e = np.zeros(M, dtype=np.int64)
        nz = top > 0
        e[nz] = np.clip(np.frexp(top[nz])[1] - 1 - 2 + 127, 0, 254)  # frexp's mantissa lies in [1/2, 1)
        q = np.abs(np.ldexp(x, (127 - e)[:, None]))
        c = nearest_e2m1(q) | (np.signbit(x).astype(np.uint8) << 3)
        c[~finite] = 0
        e[~finite] = 255
        scales[:, b] = e
        for i in range(c.shape[1]):
            k = b * BLOCK + i
            codes[:, k // 2] |= c[:, i] << (4 * (k % 2))
    return codes, scales


def nearest_e2m1(q):
    """Index of the e2m1 number nearest to each q >= 0: the distance decides, then the even index."""
    d = np.abs(np.asarray(q)[..., None] - E2M1)
    best = d.min(-1, keepdims=True)
    near = d == best
    even = near & (np.arange(8) % 2 == 0)
    return np.where(even.any(-1), even.argmax(-1), near.argmax(-1)).astype(np.uint8)


def mx4_values_ref(codes, scales, K):
    """The float64 numbers of an mx4 matrix; NaN where the exponent byte is 255."""
    M = codes.shape[0]
    out = np.zeros((M, K))
    for k in range(K):
        c = (codes[:, k // 2] >> (4 * (k % 2))) & 15
        e = scales[:, k // BLOCK].astype(np.int64)
        v = np.ldexp(np.where(c >= 8, -1.0, 1.0) * E2M1[c & 7], e - 127)
        out[:, k] = np.where(e == 255, np.nan, v)
    return out


def product_ref(X, W):
    """X W^T and the sum of the products' magnitudes, both [M, N]."""
    return X @ W.T, np.abs(X) @ np.abs(W).T


def experts_linear_ref(X, W, offsets, rows=None, R=None):
    """Y[r] = X[rows[r]] W_e^T and the products' magnitudes [R, N]; NaN on rows of no expert.

    A row index outside X counts as a row of zeros; offsets past R as R."""
    R = (len(rows) if rows is not None else X.shape[0]) if R is None else R
    Y = np.full((R, W.shape[1]), np.nan)
    B = np.full((R, W.shape[1]), np.nan)
    for e in range(W.shape[0]):
        for r in range(min(offsets[e], R), min(offsets[e + 1], R)):
            src = r if rows is None else rows[r]
            x = X[src] if 0 <= src < X.shape[0] else np.zeros(X.shape[1])
            y, b = product_ref(x[None], W[e])
            Y[r], B[r] = y[0], b[0]
    return Y, B


def route_ref(logits, k, renormalize=True):
    """ids, weights, offsets, rows, pos of float logits [T, E]."""
    T, E = logits.shape
    ids = np.full((T, k), -1, dtype=np.int32)
    weights = np.zeros((T, k))
    for t in range(T):
        l = logits[t].astype(np.float64)
        ok = [e for e in range(E) if not np.isnan(l[e]) and l[e] != -np.inf]
        order = sorted(ok, key=lambda e: (-l[e], e))[:k]
        if not order:
            continue
        top = l[order[0]]

        def w(e):
            return 1.0 if l[e] == top else np.exp(l[e] - top)

        total = sum(w(e) for e in (order if renormalize else ok))
        for j, e in enumerate(order):
            ids[t, j] = e
            weights[t, j] = w(e) / total
    offsets = np.zeros(E + 1, dtype=np.int32)
    rows = np.full(T * k, -1, dtype=np.int32)
    pos = np.full((T, k), -1, dtype=np.int32)
    r = 0
    for e in range(E):
        for t in range(T):
            for j in range(k):
                if ids[t, j] == e:
                    rows[r] = t
                    pos[t, j] = r
                    r += 1
        offsets[e + 1] = r
    return ids, weights, offsets, rows, pos


def combine_ref(O, pos, weights):
    """sum_j weights[t, j] O[pos[t, j]] and the sum of the magnitudes, over the pos that name a row."""
    T, k = pos.shape
    Y = np.zeros((T, O.shape[1]))
    B = np.zeros((T, O.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= pos[t, j] < O.shape[0]:
                Y[t] += weights[t, j] * O[pos[t, j]]
                B[t] += abs(weights[t, j]) * np.abs(O[pos[t, j]])
    return Y, B
