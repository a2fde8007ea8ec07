"""The fp8b format's calls refuse outputs at an operand's address (host only: the
refusal comes before any HIP call, and a call without rows has nothing to
refuse)."""

import pytest

import sparse_dense_gemm_amd as sdg

OK, EINVAL = sdg.SPENSE_OK, sdg.SPENSE_EINVAL
P, Q, S = 1 << 20, 1 << 21, 1 << 22  # never dereferenced


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("x,codes,scales", [(P, P, S), (P, Q, P), (P, Q, Q)])
def test_quantize(x, codes, scales, rows):
    for t in (sdg.DT_F32, sdg.DT_BF16):
        assert sdg._lib().spense_quantize_fp8b(x, t, 4, 300, 300, rows, codes, 600, scales, 3, None) == EINVAL
        assert sdg._lib().spense_quantize_fp8b(x, t, 0, 300, 300, rows, codes, 600, scales, 3, None) == OK


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("y", [Q, S])
def test_dequantize(y, rows):
    for t in (sdg.DT_F32, sdg.DT_BF16):
        assert sdg._lib().spense_dequantize_fp8b(Q, 1200, S, 3, rows, 4, 300, y, t, 300, None) == EINVAL
        assert sdg._lib().spense_dequantize_fp8b(Q, 1200, S, 3, rows, 0, 300, y, t, 300, None) == OK
