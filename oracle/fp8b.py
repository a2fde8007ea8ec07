"""Oracle of the block-scaled e4m3 format (fp8b), the products with it and the
pass between two blocks: plain NumPy, from the definitions.

An fp8b value is an e4m3fn number times the fp32 scale of its block of ``rows``
x 128.  Both quotients of the quantisation are fp32 numbers by definition
(NumPy's division rounds correctly); everything else is float64.
"""

from __future__ import annotations

import numpy as np

BLOCK8 = 128
TOP8 = np.float32(448.0)


def e4m3_values():
    """The number of each of the 256 codes (NaN for 0x7F and 0xFF)."""
    v = np.zeros(256)
    for c in range(256):
        sign, e, m = -1.0 if c & 128 else 1.0, (c >> 3) & 15, c & 7
        if e == 15 and m == 7:
            v[c] = np.nan
        else:
            v[c] = sign * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return v


def nearest_e4m3(q):
    """Code of the e4m3 number nearest to each q: the distance decides, then the even code; the sign is q's."""
    q = np.asarray(q, dtype=np.float64)
    pos = e4m3_values()[:127]  # ascending
    m = np.minimum(np.abs(q), 448.0)
    hi = np.clip(np.searchsorted(pos, m), 1, 126)
    lo = hi - 1
    below, above = m - pos[lo], pos[hi] - m
    code = np.where(below < above, lo, np.where(above < below, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code | np.where(np.signbit(q), 128, 0)).astype(np.uint8)


def fp8b_quantize_ref(X, rows=1):
    """Codes [M, K] and scales float32 [ceil(M / rows), ceil(K / 128)] of float32 X [M, K]."""
    X = np.asarray(X, dtype=np.float32)
    M, K = X.shape
    codes = np.zeros((M, K), dtype=np.uint8)
    scales = np.zeros((-(-M // rows), -(-K // BLOCK8)), dtype=np.float32)
    with np.errstate(under="ignore"):
        for i in range(scales.shape[0]):
            for b in range(scales.shape[1]):
                at = np.s_[i * rows:(i + 1) * rows, b * BLOCK8:(b + 1) * BLOCK8]
                x = X[at]
                if not np.isfinite(x).all():
                    scales[i, b] = np.nan
                    continue
                s = np.float32(np.abs(x).max() / TOP8)
                scales[i, b] = s if s > 0 else 1.0
                codes[at] = nearest_e4m3(x / scales[i, b])
    return codes, scales


def fp8b_values_ref(codes, scales, rows=1):
    """The float64 numbers of an fp8b matrix."""
    M, K = codes.shape
    i, b = np.arange(M) // rows, np.arange(K) // BLOCK8
    return e4m3_values()[codes] * scales.astype(np.float64)[i][:, b]


def fp8b_expert_values_ref(codes, scales, glu):
    """The float64 weights [E, N, K] of fp8b experts: codes [E, N, K], scales [E, blocks, ...]."""
    out = []
    for c, s in zip(codes, scales):
        if not glu:
            out.append(fp8b_values_ref(c, s, BLOCK8))
            continue
        half, nb = c.shape[0] // 2, s.shape[0] // 2
        out.append(np.concatenate([fp8b_values_ref(c[:half], s[:nb], BLOCK8), fp8b_values_ref(c[half:], s[nb:], BLOCK8)]))
    return np.stack(out)


def dropped_bits_ref(x, w):
    """Bound [M, N] on what sums of eight products at a time lose that keep 13 bits below the largest of the eight:
    8 * 2^-13 of it, over the groups of eight consecutive columns; x [M, K], w [N, K] the operands' values."""
    K = x.shape[1]
    pad = -K % 8
    x, w = (np.pad(np.abs(v), ((0, 0), (0, pad))).reshape(v.shape[0], -1, 8) for v in (x, w))
    out = np.zeros((x.shape[0], w.shape[0]))
    for g in range(x.shape[1]):
        out += (x[:, None, g] * w[None, :, g]).max(-1)
    return out * 2.0 ** -10


def block_norm_ref(O, *, eps, post=None, pre=None, gate=None, residual=None, scale=1.0, pos=None, weights=None):
    """r and y [T, H] in float64, and o (for tolerances)."""
    O = np.asarray(O, dtype=np.float64)
    if pos is not None:
        o = np.zeros((pos.shape[0], O.shape[1]))
        for t in range(pos.shape[0]):
            for j in range(pos.shape[1]):
                if 0 <= pos[t, j] < O.shape[0]:
                    o[t] += float(weights[t, j]) * O[pos[t, j]]
    else:
        o = O
    b = o / np.sqrt((o * o).mean(1, keepdims=True) + eps) * post if post is not None else o
    if gate is not None:
        b = b * gate
    r = b if residual is None else scale * np.asarray(residual, dtype=np.float64) + b
    y = r / np.sqrt((r * r).mean(1, keepdims=True) + eps)
    if pre is not None:
        y = y * pre
    return r, y, o
