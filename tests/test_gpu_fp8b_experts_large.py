"""Few rows of experts whose weights are more than the last-level cache keeps: the
calls that stream them, on both sides of the rule that decides it.

Streaming starts above 96 MiB of the weights that may be read (at most as many
experts as there are rows, counted in sixteens) and ends at 8 rows an m-tile for
each of them: 128, 256 and 512 rows of 16 experts in configurations of one, two
and four m-tiles.  Sampled columns are compared with the oracle within the
tolerances of test_gpu_fp8b_experts.py; rows behind the last group and columns
behind the row stay as they were."""

import numpy as np
import pytest
import torch

import oracle
import sparse_dense_gemm_amd as sdg

from fp8b_util import assert_close, f64
from test_gpu_fp8b_experts import reference

pytestmark = pytest.mark.gpu

E, I, K = 16, 1600, 5120
COLUMNS = np.r_[0:9, 60:68, 125:130, 1590:1600]


class Layer:
    def __init__(self, glu, I):
        g = torch.Generator("cuda").manual_seed(5)
        parts, self.glu, self.I = (2 if glu else 1), glu, I
        b = -(-I // 128)
        c = torch.empty((E, parts * I, K), dtype=torch.uint8, device="cuda")
        s = torch.empty((E, parts * b, K // 128), device="cuda")
        for e in range(E):
            for p in range(parts):
                sdg.spense_quantize_fp8b(0.02 * torch.randn(I, K, device="cuda", generator=g), c[e, p * I:(p + 1) * I],
                                         s[e, b * p:b * (p + 1)], rows=128)
        self.layer = sdg.SpenseExpertsFp8b(c, s, glu=glu)
        assert self.layer.info["device_bytes"] > 96 << 20
        n = COLUMNS
        self.W = np.concatenate([oracle.e4m3_values()[c[:, p * I + n].cpu().numpy()]
                                 * np.repeat(s[:, b * p + n // 128].double().cpu().numpy(), 128, 2) for p in range(parts)], 1)


@pytest.fixture(scope="module", params=[True, False], ids=["glu", "plain"])
def layer(request):
    h = Layer(request.param, I if request.param else 2 * I)
    yield h
    h.layer.close()


def groups(R, seed):
    """Offsets of skewed groups of R rows, some of no rows, and rows behind the last one."""
    rng = np.random.default_rng(seed)
    of = np.sort(rng.choice(E, R, p=(lambda w: w / w.sum())(np.exp(1.5 * rng.standard_normal(E)))))
    return np.concatenate([[0], np.cumsum(np.bincount(of, minlength=E))]).astype(np.int32)


CASES = [(1, None), (5, None), (13, None), (17, None), (26, None), (80, None), (128, None), (129, None),
         (26, "0"), (128, "0"), (129, "0"), (26, "1"), (256, "1"), (257, "1"), (26, "2"), (512, "2"), (513, "2")]


@pytest.mark.parametrize("kind", ["bf16", "call", "codes"])
@pytest.mark.parametrize("R,forced", CASES)
def test_few_rows_of_large_weights(layer, R, forced, kind, monkeypatch):
    if forced:
        monkeypatch.setenv("SPENSE_FP8B", forced)
    M, behind = max(2, R // 2), 3
    g = torch.Generator("cuda").manual_seed(R)
    X = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    q, s = torch.empty((M, K), dtype=torch.uint8, device="cuda"), torch.empty((M, K // 128), device="cuda")
    sdg.spense_quantize_fp8b(X, q, s)
    x = f64(X) if kind == "bf16" else oracle.fp8b_values_ref(q.cpu().numpy(), s.cpu().numpy())
    off = groups(R, R)
    rows = torch.randint(0, M, (R + behind,), device="cuda", generator=g).int()
    if R > 4:
        rows[2] = -1  # zeros
    off_d = torch.from_numpy(off).cuda()
    for yt in (torch.float32, torch.bfloat16):
        store = torch.full((R + behind, layer.I + 4), 5.0, dtype=yt, device="cuda")
        Y = store[:, :layer.I]
        if kind == "codes":
            layer.layer.quantized(q, s, off_d, Y, rows=rows)
        else:
            layer.layer(X, off_d, Y, rows=rows, adtype=sdg.DT_FP8 if kind == "call" else sdg.DT_BF16)
        assert (store[R:] == 5.0).all() and (store[:, layer.I:] == 5.0).all()
        ref, tol = reference(layer.W, x, off, rows[:R].cpu().numpy(), R, layer.glu, kind != "bf16", yt)
        assert_close(f64(Y[:R, COLUMNS]), ref, tol, (R, forced, kind, yt))
        assert not Y[:R].isnan().any()
