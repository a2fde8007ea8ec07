"""GPU parity of spense_experts_linear where X has many more rows than the call
uses: a few picked ones, or the first ones of a larger grouped matrix.
Tolerances as in test_gpu_experts."""

import numpy as np
import pytest
import torch

import sparse_dense_gemm_amd as sdg
from test_gpu_experts import KINDS, check, experts_case, offsets_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("w,a", KINDS, ids=lambda k: k)
@pytest.mark.parametrize("K", [96, 130])
@pytest.mark.parametrize("sizes", [[1], [0, 5, 0, 1], [20, 0, 17]], ids=lambda s: "x".join(map(str, s)))
def test_few_rows_of_a_large_x(sizes, K, w, a):
    E, N, M, R = len(sizes), 40, 700, sum(sizes) + 2
    rng = np.random.default_rng(K + R)
    h, W = experts_case(E, N, K, sdg.DT_MX4 if w == "mx4" else sdg.DT_BF16, False, E)
    ad = sdg.DT_MX4 if a == "mx4" else sdg.DT_BF16
    base = torch.full((M, K + 5), float("nan"), dtype=torch.bfloat16, device="cuda")
    for start in (0, 3):                                   # aligned alike or laid out first
        X = base[:, start:start + K]
        X[:] = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).cuda().bfloat16()
        rows = rng.integers(0, M, R)
        rows[0] = M - 1
        if R > 4:
            rows[1] = rows[2] = 5                          # one row for two experts or places
            rows[3] = -7
            rows[4] = M
        check(h, W, X, offsets_of(sizes), rows, R, False, ad, label=(sizes, K, w, a, start))
        X[R:] = float("nan")                               # rows that no group holds are not read
        check(h, W, X, offsets_of(sizes), None, R, False, ad, label=(sizes, K, w, a, start, "grouped"))
    h.close()
