"""spense_block_norm refuses every output at the address of an input or of another
output, but the sum in the residual's place (host only: a refusal comes before
any HIP call, and a call without rows has nothing to refuse)."""

import ctypes
import itertools

import pytest

import sparse_dense_gemm_amd as sdg

OK, EINVAL = sdg.SPENSE_OK, sdg.SPENSE_EINVAL
OUTS, INS = ("residual_out", "Y", "yscales"), ("O", "pos", "weights", "post", "pre", "gate", "residual")
AT = {name: (1 << 20) + (i << 16) for i, name in enumerate(OUTS + INS)}  # never dereferenced
PAIRS = [p for p in itertools.product(OUTS, INS) if p != ("residual_out", "residual")] + list(itertools.combinations(OUTS, 2))


def norm(T, **kw):
    args = dict(T=T, H=300, ldo=300, O_rows=8, k=2, ldg=0, ldr=300, ldro=300, ldy=300, lds=3, otype=0, wtype=0, gtype=0,
                rtype=0, ytype=sdg.DT_FP8, scale=1.0, eps=1e-6, **AT)
    args.update(kw)
    return sdg._lib().spense_block_norm(ctypes.byref(sdg.NormCall(**args)), None)


@pytest.mark.parametrize("out,other", PAIRS, ids=lambda p: p)
def test_the_same_address(out, other):
    assert norm(3, **{out: AT[other]}) == EINVAL
    assert norm(0, **{out: AT[other]}) == OK


def test_without_pos():
    assert norm(3, pos=None, weights=None, yscales=AT["gate"]) == EINVAL
    assert norm(3, pos=None, weights=None, yscales=AT["residual_out"]) == EINVAL


def test_what_may_be_the_same():
    # inputs may be one another, and types are looked at after the addresses: a bad one tells that they have passed
    for kw in (dict(), dict(residual_out=AT["residual"]), dict(post=AT["pre"], gate=AT["pre"]), dict(residual=AT["O"]),
               dict(residual_out=None), dict(residual=None, gate=None, post=None, pre=None)):
        assert norm(3, otype=9, **kw) == EINVAL
        assert norm(3, otype=sdg.DT_FP8, **kw) == sdg.SPENSE_EUNSUPPORTED, kw
