"""The router over several blocks of tokens (its second kernel joins their
counts), with masked tokens, both types, any number of experts, and more choices
in a block than LDS holds.

The reference works on whole arrays in 64 bits and is checked against the
oracle.  Whole numbers are compared exactly; a weight is within
(|l - max| + E + 8) 2^-23 of itself (see test_gpu_route)."""

import numpy as np
import pytest
import torch

import oracle
import sparse_dense_gemm_amd as sdg

T0 = 200  # tokens that the reference is checked on


def reference(l, k, renormalize):
    T, E = l.shape
    l = np.where(np.isnan(l), -np.inf, l.astype(np.float64))
    order = np.argsort(-l, axis=1, kind="stable")[:, :k]
    v = np.take_along_axis(l, order, 1)
    none = v == -np.inf
    with np.errstate(invalid="ignore"):
        p, every = (np.where(a == v[:, :1], 1.0, np.exp(a - v[:, :1])) for a in (v, l))
    p = np.where(none, 0.0, p)
    total = p.sum(1, keepdims=True) if renormalize else np.where(l == -np.inf, 0.0, every).sum(1, keepdims=True)
    weights = p / np.where(total > 0, total, 1.0)
    ids = np.where(none, -1, order).astype(np.int32)
    flat = np.where(none, E, order).ravel()
    at = np.argsort(flat, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E + 1)[:E])]).astype(np.int32)
    have = offsets[E]
    rows = np.full(T * k, -1, dtype=np.int32)
    rows[:have] = at[:have] // k
    pos = np.full(T * k, -1, dtype=np.int32)
    pos[at[:have]] = np.arange(have)
    with np.errstate(invalid="ignore"):
        d = np.where(none, 0.0, v[:, :1] - v)
    return ids, weights, offsets, rows, pos.reshape(T, k), np.where(np.isfinite(d), d, 0.0)


def logits(T, E, seed):
    """Random logits, some experts more popular, some off; some tokens with few experts left or none."""
    rng = np.random.default_rng(seed)
    l = (rng.standard_normal((T, E)) * 2 + rng.standard_normal(E)).astype(np.float32)
    l[rng.random((T, E)) < 0.3] = -np.inf
    few = rng.random(T) < 0.05
    l[few, 1:] = -np.inf
    l[rng.random(T) < 0.03] = -np.inf
    l[rng.random(T) < 0.02] = np.nan
    l[rng.random((T, E)) < 0.01] = np.inf
    l[::5] = np.round(l[::5])  # ties
    return l


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("E,k", [(8, 2), (17, 17), (40, 5)])
def test_reference(E, k, renormalize):
    l = logits(T0, E, E)
    for got, want in zip(reference(l, k, renormalize), oracle.route_ref(l, k, renormalize)):
        assert np.allclose(got, want, rtol=1e-12, atol=0)


# several blocks from 257 tokens on; 32 to 1024 tokens a block
@pytest.mark.gpu
@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,k", [
    (257, 1, 1), (300, 8, 8), (1000, 17, 2), (1025, 60, 20), (4097, 128, 8), (700, 300, 20), (513, 600, 17),
    (290, 1024, 20), (9000, 1024, 4), (20011, 64, 64), (40000, 48, 20), (70001, 16, 3),
])
def test_blocks(T, E, k, renormalize, bf16):
    L = torch.from_numpy(logits(T, E, T + E)).cuda()
    L = L.bfloat16() if bf16 else L
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, pos = torch.full((T, k), 77, **i32), torch.full((T, k), 77, **i32)
    weights = torch.full((T, k), 7.0, device="cuda")
    offsets, rows = torch.full((E + 1,), 77, **i32), torch.full((T * k,), 77, **i32)
    need = sdg.spense_route_workspace(T, E, k)
    assert need > 0
    work = torch.full((need,), 0x5A, dtype=torch.uint8, device="cuda")
    sdg.spense_route(L, k, ids, weights, offsets, rows, pos, work, renormalize=renormalize)
    got = [t.cpu().numpy() for t in (ids, weights, offsets, rows, pos)]
    *want, d = reference(L.float().cpu().numpy(), k, renormalize)
    for name, g, w in zip(("ids", "weights", "offsets", "rows", "pos"), got, want):
        if name == "weights":
            assert (np.abs(g - w) <= (d + E + 8) * 2.0 ** -23 * w + 1e-37).all()
        else:
            assert np.array_equal(g, w), name
