"""The binding of the mx4, experts' and router entry points refuses tensors that
the call would read or write wrongly, and takes all others.  Runs on CPU tensors
with the library's host code and a runtime that launches nothing."""

import pytest
import torch

import host_library
import sparse_dense_gemm_amd as sdg

E, N, K, T, k = 4, 32, 64, 6, 2
R = T * k
F32, BF16, I32, I64, U8 = torch.float32, torch.bfloat16, torch.int32, torch.int64, torch.uint8


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    return host_library.build(tmp_path_factory.mktemp("host"))


@pytest.fixture(autouse=True)
def binding(host, monkeypatch):
    monkeypatch.setattr(sdg, "LIB_PATH", host)
    monkeypatch.setattr(sdg, "_lib_handle", None)


def every_other(t):
    """The same values, not contiguous along the last dimension."""
    return t.repeat_interleave(2, -1)[..., ::2]


def refuses(call, base, **bad):
    for name, value in bad.items():
        with pytest.raises((TypeError, ValueError)):
            call(**{**base, name: value})
            pytest.fail(f"{name} {value.dtype} {tuple(value.shape)} was taken")


def mx4_layer():
    return sdg.SpenseLinearMx4(torch.zeros((N, K // 2), dtype=U8), torch.zeros((N, K // 32), dtype=U8), stream=0)


def experts(**kw):
    return sdg.SpenseExperts(torch.zeros((E, N, K), dtype=BF16), stream=0, **kw)


@pytest.mark.parametrize("form", ["layer", "handle"])
def test_linear_w4a4(form):
    layer = mx4_layer()

    def call(X, Y):
        if form == "layer":
            layer.w4a4(X, Y, stream=0)
        else:
            sdg.spense_linear_w4a4(layer.handle, X, Y, stream=0)

    X, Y = torch.zeros((T, K), dtype=BF16), torch.zeros((T, N))
    call(X, Y)
    call(X.repeat(1, 2)[:, 3:K + 3], Y.repeat(1, 2)[:, :N])     # rows of a larger matrix
    call(X, torch.zeros((T + 1, N), dtype=BF16))
    for bad in (X.float(), X.view(torch.int16), X.half(), every_other(X), X.repeat(1, 2)[:, :K - 1], X[0]):
        refuses(call, dict(X=X, Y=Y), X=bad)
    for bad in (Y[:-1], every_other(Y), Y.repeat(1, 2)[:, :N - 1], Y.to(I32), Y.double()):
        refuses(call, dict(X=X, Y=Y), Y=bad)
    with pytest.raises(ValueError):
        sdg.spense_linear_w4a4(layer.handle, X, torch.zeros((T + 1, N)), M=T + 1, stream=0)


def test_mx4_layer_call():
    layer = mx4_layer()
    X, Y = torch.zeros((T, K), dtype=BF16), torch.zeros((T, N))

    def call(X, Y):
        layer(X, Y, stream=0)

    call(X, Y)
    for bad in (every_other(X), X.repeat(1, 2)[:, :K - 1]):
        refuses(call, dict(X=X, Y=Y), X=bad)
    for bad in (Y[:-1], every_other(Y)):
        refuses(call, dict(X=X, Y=Y), Y=bad)


@pytest.mark.parametrize("form", ["layer", "handle"])
@pytest.mark.parametrize("glu", [False, True])
def test_experts_linear(form, glu):
    layer = experts(glu=glu)
    cols = N // 2 if glu else N

    def call(X, offsets, Y, rows):
        if form == "layer":
            layer(X, offsets, Y, rows=rows, stream=0)
        else:
            sdg.spense_experts_linear(layer.handle, X, offsets, Y, rows=rows, stream=0)

    base = dict(X=torch.zeros((T, K), dtype=BF16), offsets=torch.zeros(E + 1, dtype=I32), Y=torch.zeros((R, cols)),
                rows=torch.zeros(R, dtype=I32))
    call(**base)
    call(**{**base, "rows": None, "X": torch.zeros((R, K), dtype=BF16)})
    call(**{**base, "offsets": torch.zeros(E + 9, dtype=I32), "rows": torch.zeros(R + 5, dtype=I32)})
    X, offsets, Y, rows = base.values()
    for bad in (X.float(), X.half(), every_other(X), X.repeat(1, 2)[:, :K - 1], X[0]):
        refuses(call, base, X=bad)
    for bad in (offsets.to(I64), offsets.float(), offsets[:-1], every_other(offsets)):
        refuses(call, base, offsets=bad)
    for bad in (rows.to(I64), rows[:-1], every_other(rows)):
        refuses(call, base, rows=bad)
    for bad in (every_other(Y), Y.repeat(1, 2)[:, :cols - 1], Y.double(), Y[:, 0]):
        refuses(call, base, Y=bad)
    with pytest.raises(ValueError):
        sdg.spense_experts_linear(layer.handle, X, offsets, Y, rows=torch.zeros(R + 1, dtype=I32), R=R + 1, stream=0)


def test_route():
    def call(**kw):
        sdg.spense_route(k=k, stream=0, **kw)

    base = dict(logits=torch.zeros((T, E)), ids=torch.zeros((T, k), dtype=I32), weights=torch.zeros((T, k)),
                offsets=torch.zeros(E + 1, dtype=I32), rows=torch.zeros(R, dtype=I32),
                pos=torch.zeros((T, k), dtype=I32))
    call(**base)
    call(**{**base, "logits": torch.zeros((T, 3 * E), dtype=BF16)[:, 5:5 + E]})
    for name in ("ids", "offsets", "rows", "pos"):
        t = base[name]
        for bad in (t.to(I64), t.to(torch.int16), t.float(), every_other(t), t.flatten()[:-1]):
            refuses(call, base, **{name: bad})
    for bad in (base["weights"].bfloat16(), base["weights"].double(), every_other(base["weights"])):
        refuses(call, base, weights=bad)
    for bad in (every_other(base["logits"]), base["logits"].half(), base["logits"].t().contiguous().t()):
        refuses(call, base, logits=bad)


def test_combine():
    def call(**kw):
        sdg.spense_experts_combine(stream=0, **kw)

    base = dict(O=torch.zeros((R, N)), pos=torch.zeros((T, k), dtype=I32), weights=torch.zeros((T, k)),
                Y=torch.zeros((T, N), dtype=BF16))
    call(**base)
    call(**{**base, "O": torch.zeros((3, N + 7), dtype=BF16), "Y": torch.zeros((T + 2, N))})
    for bad in (base["pos"].to(I64), every_other(base["pos"]), base["pos"].float()):
        refuses(call, base, pos=bad)
    for bad in (base["weights"].bfloat16(), base["weights"][:-1], every_other(base["weights"])):
        refuses(call, base, weights=bad)
    for bad in (every_other(base["O"]), base["O"].repeat(1, 2)[:, :N - 1], base["O"].double(), base["O"][0]):
        refuses(call, base, O=bad)
    for bad in (base["Y"][:-1], every_other(base["Y"]), base["Y"].double()):
        refuses(call, base, Y=bad)


def test_quantize_and_dequantize():
    c, s = torch.zeros((T, K // 2), dtype=U8), torch.zeros((T, K // 32), dtype=U8)
    for call in (lambda x, **kw: sdg.spense_quantize_mx4(x, c, s, stream=0, **kw),
                 lambda x, **kw: sdg.spense_dequantize_mx4(c, s, x, stream=0, **kw)):
        x = torch.zeros((T, K))
        call(x)
        call(x.repeat(1, 2)[:, 5:5 + K].bfloat16())
        for bad in (every_other(x), x.t().contiguous().t(), x.half(), x.double()):
            refuses(lambda x: call(x), dict(x=x), x=bad)
    call = sdg.spense_quantize_mx4
    call(torch.zeros((T, K), dtype=torch.int16), c, s, xdtype=sdg.DT_BF16, stream=0)   # storage of a named type
    with pytest.raises(TypeError):
        call(torch.zeros((T, K), dtype=BF16), c, s, xdtype=sdg.DT_F32, stream=0)
    with pytest.raises(TypeError):
        sdg.spense_dequantize_mx4(c, s, torch.zeros((T, K), dtype=BF16), ydtype=sdg.DT_F32, stream=0)


def test_pack_experts():
    W = torch.zeros((E, N, K), dtype=BF16)
    sdg.SpenseExperts(W, stream=0)
    sdg.SpenseExperts(W.view(torch.int16), sdg.DT_BF16, stream=0)
    sdg.SpenseExperts(W.repeat(1, 1, 2)[..., :K], K=K - 1, stream=0)
    for bad, kw in ((W.view(torch.int16).to(U8), {}), (W.repeat(1, 1, 2)[..., :K - 1], dict(K=K)), (W.float(), {})):
        with pytest.raises((TypeError, ValueError)):
            sdg.spense_pack_experts(bad, sdg.DT_BF16, stream=0, **kw)


def test_w8a8_takes_bf16_only():
    h = sdg.spense_pack(torch.zeros((N, K), dtype=U8), scales=torch.ones(N), dense_fraction=0.0, stream=0)
    X, Y = torch.zeros((T, K), dtype=BF16), torch.zeros((T, N))
    sdg.spense_linear_w8a8(h, X, Y, stream=0)
    for bad in (X.float(), X.half()):
        with pytest.raises(TypeError):
            sdg.spense_linear_w8a8(h, bad, Y, stream=0)
    sdg.spense_free(h)


def test_nothing_to_do():
    """Calls without rows: torch's empty tensors have no address."""
    c, s = torch.zeros((0, K // 2), dtype=U8), torch.zeros((0, K // 32), dtype=U8)
    assert c.data_ptr() == 0
    sdg.spense_quantize_mx4(torch.zeros((0, K)), c, s, stream=0)
    sdg.spense_dequantize_mx4(c, s, torch.zeros((0, K), dtype=BF16), stream=0)
    no_pairs, offsets = torch.zeros((0, k), dtype=I32), torch.zeros(E + 1, dtype=I32)
    for X in (torch.zeros((0, K), dtype=BF16), torch.zeros((T, K), dtype=BF16)):
        experts()(X, offsets, torch.zeros((0, N)), stream=0)
        experts()(X, offsets, torch.zeros((0, N)), rows=torch.zeros(0, dtype=I32), stream=0)
    sdg.spense_route(torch.zeros((0, E)), k, no_pairs, torch.zeros((0, k)), offsets, torch.zeros(0, dtype=I32),
                     no_pairs, stream=0)
    for O in (torch.zeros((0, N)), torch.zeros((R, N))):
        sdg.spense_experts_combine(O, no_pairs, torch.zeros((0, k)), torch.zeros((0, N)), stream=0)
    # tokens whose experts gave no rows
    sdg.spense_experts_combine(torch.zeros((0, N)), torch.zeros((T, k), dtype=I32), torch.zeros((T, k)),
                               torch.zeros((T, N)), stream=0)
