"""GPU parity of spense_block_norm against the oracle.

Tolerances.  A mean of squares sums at most 32 squares a thread one after the
other, then over 64 lanes and 16 waves in 16 more additions, each off by 2^-24 of the
sum (all terms positive), more in a row longer than 32768 columns, whose threads
go on in the same way: n = 32 ceil(H / 32768) + 24 steps, half of that for
the root, with the division by H, eps, and the root instruction (2^-23) another
2^-22: rel = n 2^-25 + 2^-22 for a factor 1 / sqrt(mean + eps).
o is off by k 2^-24 sum |w O|; b = o inv post gate by that times |inv post gate|
and by (rel + 3 2^-24) |b|; r by 2^-24 |r| more, and 2^-24 of the residual's
part.  y = r inv' pre: r's error times |inv' pre|, the change of inv' that r's
error brings (at most its rms over r's), and (rel + 2 2^-24) |y|."""

import numpy as np
import pytest
import torch

import oracle
import sparse_dense_gemm_amd as sdg

from fp8b_util import TYPES, assert_close, dev, f64

pytestmark = pytest.mark.gpu

EPS = 1e-6


def tensors(T, H, seed, o="f32", r="f32", w="f32", g="f32", k=0, gate=None, post=True, pre=True, residual=True):
    rng = np.random.default_rng(seed)

    def t(shape, ty, f=lambda a: a):
        return dev(f(rng.standard_normal(shape)).astype(np.float32)).to(TYPES[ty])

    d = dict(O=t((T if not k else max(T * k, 1), H), o, lambda a: a * np.exp(rng.standard_normal((a.shape[0], 1)))))
    if k:
        d["pos"] = dev(rng.permutation(T * k).astype(np.int32).reshape(T, k))
        d["weights"] = dev(rng.random((T, k)).astype(np.float32))
    if residual:
        d["residual"] = t((T, H), r, lambda a: 3 * a)
    if post:
        d["post"] = t((H,), w, lambda a: 1 + 0.2 * a)
    if pre:
        d["pre"] = t((H,), w, lambda a: 1 + 0.2 * a)
    if gate:
        d["gate"] = t((T, H) if gate == "token" else (1, H) if gate == "row" else (H,), g, np.tanh)
    return d


def reference(d, scale, eps=EPS):
    """r, y and their tolerances before the outputs' roundings."""
    n = {k: (v.cpu().numpy() if k == "pos" else f64(v)) for k, v in d.items()}
    O = n.pop("O")
    r, y, o = oracle.block_norm_ref(O, eps=eps, scale=scale, **n)
    T, H = r.shape
    rel = (32 * -(-H // 32768) + 24) * 2.0 ** -25 + 2.0 ** -22
    do = 0.0
    if "pos" in n:
        _, _, mags = oracle.block_norm_ref(np.abs(O), eps=eps, pos=n["pos"], weights=np.abs(n["weights"]))
        do = n["pos"].shape[1] * 2.0 ** -24 * mags
    gate = n.get("gate", 1.0)
    if "post" in n:
        inv = 1 / np.sqrt((o * o).mean(1, keepdims=True) + eps)
        f = np.abs(inv * n["post"] * gate)
    else:
        f = np.abs(gate) * np.ones((1, H))
    b = np.abs(o) * f
    # the change of inv that o's error brings: at most its rms over o's rms
    drms = np.sqrt((np.square(do * np.ones_like(o))).mean(1, keepdims=True) / ((o * o).mean(1, keepdims=True) + eps))
    dr = do * f + ((rel + drms if "post" in n else 0.0) + 3 * 2.0 ** -24) * b + 2.0 ** -23 * np.abs(r)
    if "residual" in n:
        dr = dr + 2.0 ** -24 * np.abs(scale * n["residual"])
    m = (r * r).mean(1, keepdims=True) + eps
    inv2 = np.abs(n.get("pre", 1.0)) / np.sqrt(m)
    dy = dr * inv2 + (rel + 2 * 2.0 ** -24 + np.sqrt((dr * dr).mean(1, keepdims=True) / m)) * np.abs(y)
    return r, y, dr, dy


def run(d, rt, y, T, H, scale=0.75, eps=EPS, store_r=True, pad=0, inplace=False):
    """residual_out and Y (codes and scales for "fp8"); columns and rows behind them stay as they are."""
    d = dict(d)
    O, residual = d.pop("O"), d.pop("residual", None)
    R2 = None
    if store_r:
        R2s = residual if inplace else torch.full((T + 1, H + pad), 5.0, dtype=TYPES[rt], device="cuda")
        R2 = R2s if inplace else R2s[:T, :H]
    Y = ys = Ys = None
    if y == "fp8":
        Ys = torch.full((T + 1, H + pad), 0x5A, dtype=torch.uint8, device="cuda")
        S = torch.full((T + 1, -(-H // 128) + pad), 5.0, device="cuda")
        Y, ys = Ys[:T, :H], S[:T, :-(-H // 128)]
    elif y:
        Ys = torch.full((T + 1, H + pad), 5.0, dtype=TYPES[y], device="cuda")
        Y = Ys[:T, :H]
    sdg.spense_block_norm(O, residual, R2, Y, eps=eps, scale=scale, yscales=ys, **d)
    torch.cuda.synchronize()
    if store_r and not inplace:
        assert (R2s[T] == 5.0).all() and (R2s[:, H:] == 5.0).all()
    if y:
        assert (Ys[T] == (0x5A if y == "fp8" else 5.0)).all() and (Ys[:, H:] == (0x5A if y == "fp8" else 5.0)).all()
    if y == "fp8":
        assert (S[T] == 5.0).all() and (S[:, -(-H // 128):] == 5.0).all()
    return R2, Y, ys


def check(d, rt, y, T, H, label, **kw):
    r, want, dr, dy = reference(d, 0.75)
    R2, Y, ys = run(d, rt, y, T, H, **kw)
    if R2 is not None:
        assert_close(f64(R2), r, dr + (2.0 ** -8 if rt == "bf16" else 0.0) * np.abs(r), (label, "residual"))
    if y == "fp8":
        # the same bits as quantising the unrounded y
        d2 = dict(d)
        _, Y32, _ = run(d2, rt, "f32", T, H, store_r=False)
        c, s = torch.empty((T, H), dtype=torch.uint8, device="cuda"), torch.empty((T, -(-H // 128)), device="cuda")
        sdg.spense_quantize_fp8b(Y32.contiguous(), c, s)
        assert torch.equal(c, Y) and torch.equal(s, ys), (label, "codes")
        assert_close(f64(Y32), want, dy, (label, "y of the codes"))
    elif y:
        assert_close(f64(Y), want, dy + (2.0 ** -8 if y == "bf16" else 0.0) * np.abs(want), (label, "y"))


@pytest.mark.parametrize("H", [1, 7, 8, 64, 129, 1000, 5120, 8192, 8193, 12000, 32768, 32770, 40001])
@pytest.mark.parametrize("y", ["f32", "bf16", "fp8"])
def test_lengths(H, y):
    T = 3
    for r, gate in (("f32", "row"), ("bf16", "token")):
        d = tensors(T, H, H, o="bf16", r=r, w="bf16", g="bf16", gate=gate)
        check(d, r, y, T, H, (H, y, r), pad=3)


@pytest.mark.parametrize("o", ["f32", "bf16"])
@pytest.mark.parametrize("r", ["f32", "bf16"])
@pytest.mark.parametrize("w", ["f32", "bf16"])
@pytest.mark.parametrize("gate,g", [(None, "f32"), ("vector", "bf16"), ("row", "f32"), ("token", "f32"), ("token", "bf16")])
def test_types(o, r, w, gate, g):
    T, H = 5, 712
    d = tensors(T, H, 1, o=o, r=r, w=w, g=g, gate=gate)
    for y in ("f32", "bf16", "fp8"):
        check(d, r, y, T, H, (o, r, w, gate, g, y))


@pytest.mark.parametrize("H", [520, 1003, 9000, 40003])
@pytest.mark.parametrize("k", [1, 2, 3, 5])
def test_sum_over_experts(H, k):
    """Rows picked and weighted; places outside O add nothing, whatever their weight; O may be empty."""
    T = 4
    for o in ("f32", "bf16"):
        d = tensors(T, H, k, o=o, r="bf16", k=k, post=k % 2 == 0)
        d["pos"][0, 0] = -1
        d["pos"][1] = T * k
        d["weights"][1] = float("nan")
        d["weights"][0, 0] = float("inf")
        ref = dict(d, weights=torch.where(d["weights"].isfinite(), d["weights"], torch.zeros_like(d["weights"])))
        r, want, dr, dy = reference(ref, 0.75)
        R2, Y, _ = run(d, "bf16", "f32", T, H)
        assert_close(f64(R2), r, dr + 2.0 ** -8 * np.abs(r), (H, k, o))
        assert_close(f64(Y), want, dy, (H, k, o))


def test_sum_agrees_with_combine():
    """With no norm, gate or residual it is spense_experts_combine, bit for bit."""
    T, k, H = 33, 2, 640
    d = tensors(T, H, 3, o="f32", k=k, post=False, pre=False, residual=False)
    R2 = torch.empty((T, H), device="cuda")
    sdg.spense_block_norm(d["O"], None, R2, None, eps=EPS, pos=d["pos"], weights=d["weights"])
    Y = torch.empty((T, H), device="cuda")
    sdg.spense_experts_combine(d["O"], d["pos"], d["weights"], Y)
    assert torch.equal(R2, Y)


@pytest.mark.parametrize("H", [300, 5120, 20000, 40000])
def test_parts_left_out(H):
    """No residual, no stored sum, no y, no weights, in place."""
    T = 3
    check(tensors(T, H, 2, residual=False), "f32", "bf16", T, H, "no residual")
    check(tensors(T, H, 3, post=False, gate="token"), "f32", "f32", T, H, "no norm after the block")
    check(tensors(T, H, 4, pre=False), "f32", "fp8", T, H, "no weights before the next")
    check(tensors(T, H, 5), "bf16", "fp8", T, H, "sum not stored", store_r=False)
    check(tensors(T, H, 6, r="bf16"), "bf16", None, T, H, "no y")
    for r in ("f32", "bf16"):
        d = tensors(T, H, 7, r=r, gate="row")
        R2, Y, _ = run(d, r, "bf16", T, H)
        e = dict(d, residual=d["residual"].clone())
        R3, Z, _ = run(e, r, "bf16", T, H, inplace=True)
        assert torch.equal(R3, R2) and torch.equal(Z, Y) and R3.data_ptr() == e["residual"].data_ptr()


def test_strides_and_alignment():
    """Operands that start anywhere: the same bits."""
    T, H = 6, 1024
    d = tensors(T, H, 8, o="bf16", r="bf16", w="bf16", g="bf16", gate="token")
    R2, Y, ys = run(d, "bf16", "fp8", T, H)
    for pad in (1, 3, 8):
        e = {}
        for n, v in d.items():
            if v.dim() == 1:
                s = torch.empty(H + pad, dtype=v.dtype, device="cuda")[pad:]
            else:
                s = torch.full((T, H + 2 * pad), float("nan"), dtype=v.dtype, device="cuda")[:, pad:pad + H]
            s.copy_(v)
            e[n] = s
        R3, Z, zs = run(e, "bf16", "fp8", T, H, pad=pad)
        assert torch.equal(R3, R2) and torch.equal(Z, Y) and torch.equal(zs, ys), pad


def test_zero_rows_and_non_finite_values():
    T, H = 6, 300
    d = tensors(T, H, 9, o="f32", r="f32")
    d["O"][1] = 0.0
    d["O"][2] = 0.0
    d["residual"][2] = 0.0
    d["O"][3, 5] = float("nan")
    d["O"][4, 6] = float("inf")
    R2, Y, ys = run(d, "f32", "fp8", T, H)
    r, want, dr, dy = reference({k: (v[[0, 1, 2, 5]] if v.dim() == 2 else v) for k, v in d.items()}, 0.75)
    assert_close(f64(R2[[0, 1, 2, 5]]), r, dr, "rows beside the others")
    assert (R2[2] == 0).all() and (Y[2] == 0).all() and (ys[2] == 1).all()
    assert R2[3].isnan().all() and ys[3].isnan().all() and (Y[3] == 0).all()
    assert ys[4].isnan().all() and (Y[4] == 0).all()  # 0 * inf in the norm after the block


def test_sums_of_squares_out_of_range():
    """Squares beyond the range of fp32: the mean is infinite and the normalised row 0, as in the formula."""
    T, H = 3, 256
    d = tensors(T, H, 11, post=False)
    d["O"][1] = 1e25
    R2, Y, _ = run(d, "f32", "f32", T, H)
    assert (R2[1] == fma(d, 1)).all() and (Y[1] == 0).all()
    r, want, dr, dy = reference({k: (v[[0, 2]] if v.dim() == 2 else v) for k, v in d.items()}, 0.75)
    assert_close(f64(Y[[0, 2]]), want, dy, "rows beside it")


def fma(d, t):
    """0.75 * residual + O rounded once."""
    return dev((0.75 * f64(d["residual"][t]) + f64(d["O"][t])).astype(np.float32))


def test_many_rows():
    """More rows than a wave of workgroups, streamed results: sampled rows."""
    T, H = 8191, 5120
    g = torch.Generator("cuda").manual_seed(1)
    O = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    R = 3 * torch.randn(T, H, device="cuda", generator=g)
    post, pre = (1 + 0.2 * torch.randn(H, device="cuda", generator=g) for _ in range(2))
    at = torch.tensor([0, 1, 767, 768, 4000, 8190], device="cuda")
    d = dict(O=O, residual=R, post=post, pre=pre)
    R2, Y, _ = run(d, "f32", "bf16", T, H)
    r, want, dr, dy = reference(dict(O=O[at], residual=R[at], post=post, pre=pre), 0.75)
    assert_close(f64(R2[at]), r, dr, "residual")
    assert_close(f64(Y[at]), want, dy + 2.0 ** -8 * np.abs(want), "y")
    _, Z, zs = run(d, "f32", "fp8", T, H)
    _, Y32, _ = run(d, "f32", "f32", T, H)
    c, s = torch.empty((T, H), dtype=torch.uint8, device="cuda"), torch.empty((T, 40), device="cuda")
    sdg.spense_quantize_fp8b(Y32.contiguous(), c, s)
    assert torch.equal(c, Z) and torch.equal(s, zs)


def test_no_rows():
    e = torch.empty((0, 64), device="cuda")
    sdg.spense_block_norm(e, e, e, e, eps=EPS)
    pos = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    Y = torch.empty((2, 64), device="cuda")
    R = torch.randn((2, 64), device="cuda")
    sdg.spense_block_norm(e, R, None, Y, eps=EPS, pos=pos, weights=torch.ones((2, 2), device="cuda"))
    want = oracle.block_norm_ref(np.zeros((2, 64)), eps=EPS, residual=f64(R))[1]
    assert np.allclose(f64(Y), want, rtol=2.0 ** -18)


def test_pointers_of_an_empty_o():
    """O may be NULL where no place of pos can name a row."""
    T, H = 2, 64
    pos, w = torch.zeros((T, 1), dtype=torch.int32, device="cuda"), torch.ones((T, 1), device="cuda")
    Y = torch.full((T, H), 3.0, device="cuda")
    call = sdg.NormCall(T=T, H=H, O=None, ldo=H, O_rows=0, pos=pos.data_ptr(), weights=w.data_ptr(), k=1, otype=1,
                        residual_out=Y.data_ptr(), ldro=H, rtype=0, scale=1.0, eps=EPS)
    import ctypes
    assert sdg._lib().spense_block_norm(ctypes.byref(call), torch.cuda.current_stream().cuda_stream) == 0
    assert (Y == 0).all()


@pytest.mark.parametrize("H", [9, 10, 11, 13, 15, 63, 65, 121, 127, 130, 135, 517, 575, 8199, 9001])
@pytest.mark.parametrize("k", [0, 2])
def test_row_ends(H, k):
    """Rows that end inside a piece of eight columns, also with the residual in place and unaligned rows."""
    for y in ("f32", "bf16", "fp8"):
        d = tensors(5, H, H + k, o="bf16", r="bf16", w="bf16", gate="token", g="bf16", k=k)
        check(d, "bf16", y, 5, H, (H, k, y), pad=3)
        R2, Y, ys = run(d, "bf16", y, 5, H)
        d["residual"] = d["residual"].clone()
        S2, Z, zs = run(d, "bf16", y, 5, H, inplace=True)
        assert torch.equal(R2, S2) and torch.equal(Y, Z) and (ys is None or torch.equal(ys, zs))


@pytest.mark.parametrize("H,col", [(130, 125), (130, 127), (130, 128), (130, 121), (135, 127), (135, 128), (14, 7), (14, 8)])
@pytest.mark.parametrize("y", ["f32", "bf16", "fp8"])
def test_one_column_of_the_last_norm_stays_in_its_place(H, col, y):
    """A NaN in `pre` reaches its own column alone, or its block of codes."""
    d = tensors(3, H, 1, w="f32")
    _, want, wants = run(d, "f32", y, 3, H)
    d["pre"][col] = float("nan")
    _, Y, ys = run(d, "f32", y, 3, H)
    at = torch.arange(H, device="cuda")
    if y == "fp8":
        b = col // 128
        assert ys[:, b].isnan().all() and (Y[:, at // 128 == b] == 0).all()
        others = torch.arange(ys.shape[1], device="cuda") != b
        assert torch.equal(ys[:, others], wants[:, others]) and torch.equal(Y[:, at // 128 != b], want[:, at // 128 != b])
    else:
        assert Y[:, col].isnan().all() and torch.equal(Y[:, at != col], want[:, at != col])
