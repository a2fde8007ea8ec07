"""The 8-bit expert layer of examples/expert_block.py: norm, router, experts and
norm run together, against the oracle step by step through its own
intermediates, and as one HIP graph on a stream of its own with eager work
between the replays; the fp8b calls captured, after larger calls, on two streams
at once."""

import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle
import sparse_dense_gemm_amd as sdg

from fp8b_util import acts, assert_close, bf16, dev, f64, product_tolerance, weights
from test_gpu_fp8b_experts import reference as experts_reference
from test_gpu_block_norm import reference as norm_reference

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("expert_block", os.path.join(ROOT, "examples", "expert_block.py"))
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)

E, H, I, K, TOP = 6, 320, 136, 2, 70


def make():
    w = example.make(E, H, I)
    return w, example.ExpertLayer8(*w, example.make_norms(H), K, TOP)


def inputs(T):
    g = torch.Generator("cuda").manual_seed(T)
    return (torch.randn(T, H, device="cuda", generator=g).bfloat16(),
            (2 * torch.randn(T, H, device="cuda", generator=g)).bfloat16())


def outputs(T):
    return torch.empty((T, H), dtype=torch.uint8, device="cuda"), torch.empty((T, -(-H // 128)), device="cuda")


def values(codes, scales, rows=1):
    return oracle.fp8b_values_ref(codes.cpu().numpy(), scales.cpu().numpy(), rows)


@pytest.mark.parametrize("T", [1, 5, 70])
def test_layer(T):
    (gate_up, down, router), layer = make()
    n = layer.norms
    attention, residual = inputs(T)
    before = residual.clone()
    codes, scales = layer(attention, residual, *outputs(T))
    torch.cuda.synchronize()
    R = T * K
    # the first pass: codes within half a step (2^-4 of a value, 2^-10 of its scale) of the norm
    d = dict(O=attention, residual=before, post=n["post"], pre=n["pre"])
    r, y, dr, dy = norm_reference_scaled(d)
    s = np.repeat(layer.scales[:T].double().cpu().numpy(), 128, 1)[:, :H]
    x = values(layer.codes[:T], layer.scales[:T])
    assert_close(x, y, dy + np.maximum(2.0 ** -4 * (np.abs(y) + dy), 2.0 ** -10 * s) * (1 + 2.0 ** -20), "codes")
    # the router, on the device's own codes
    Wr = values(*example.quantized8(router), 128)
    ref, B = oracle.product_ref(x, Wr)
    assert_close(f64(layer.logits[:T]), ref, product_tolerance(x, Wr, ref, B, H, True, torch.float32), "logits")
    ids, w, off, rows, pos = oracle.route_ref(layer.logits[:T].cpu().numpy(), K)
    assert np.array_equal(layer.ids[:T].cpu().numpy(), ids) and np.array_equal(layer.rows[:R].cpu().numpy(), rows)
    assert np.array_equal(layer.offsets.cpu().numpy(), off) and np.array_equal(layer.pos[:T].cpu().numpy(), pos)
    # gate and up
    Wg = np.stack([np.concatenate([values(*example.quantized8(p), 128) for p in g.chunk(2)]) for g in gate_up])
    A, tol = experts_reference(Wg, x, off, rows, R, True, True, torch.bfloat16)
    assert_close(f64(layer.A[:R]), A, tol, "gate and up")
    # down, on the device's own intermediate, quantised in the call
    a = oracle.fp8b_values_ref(*oracle.fp8b_quantize_ref(layer.A[:R].float().cpu().numpy()))
    Wd = np.stack([values(*example.quantized8(m), 128) for m in down])
    O, tol = experts_reference(Wd, a, off, None, R, False, True, torch.float32)
    assert_close(f64(layer.O[:R]), O, tol, "down")
    # the second pass, on the residual that the first one left: r before its rounding is off by half a step more
    r1 = f64_bf16(r)
    d = dict(O=layer.O[:R], pos=layer.pos[:T], weights=layer.weights[:T], residual=dev(r1.astype(np.float32)),
             pre=n["pre_next"], gate=n["gate"])
    r2, y2, dr2, dy2 = norm_reference_scaled(d)
    slack = dr + 2.0 ** -7 * np.abs(r)  # the first residual may have rounded the other way
    assert_close(f64(residual), r2, dr2 + slack + 2.0 ** -8 * (np.abs(r2) + slack), "residual")
    m = np.sqrt((r2 * r2).mean(1, keepdims=True) + layer.eps)
    moved = slack / m * np.abs(f64(n["pre_next"])) + np.sqrt((slack * slack).mean(1, keepdims=True)) / m * np.abs(y2)
    s = np.repeat(scales.double().cpu().numpy(), 128, 1)[:, :H]
    top = dy2 + moved
    assert_close(values(codes, scales), y2, top + np.maximum(2.0 ** -4 * (np.abs(y2) + top), 2.0 ** -10 * s) * (1 + 2.0 ** -20),
                 "next codes")
    layer.close()


def f64_bf16(a):
    return f64(dev(a.astype(np.float32)).bfloat16())


def norm_reference_scaled(d):
    """The norm tests' reference at scale 1 instead of their 0.75: the residual enters it divided by that."""
    e = dict(d)
    e["residual"] = (d["residual"].float() / 0.75).double()
    n = {k: v for k, v in e.items()}
    r, y, dr, dy = norm_reference(n, 0.75, 1e-6)
    # the division rounds to 32 bits: 2^-24 of the residual more
    more = 2.0 ** -23 * np.abs(f64(d["residual"]))
    m = np.sqrt((r * r).mean(1, keepdims=True) + 1e-6)
    pre = np.abs(f64(d["pre"]))
    return r, y, dr + more, dy + more / m * pre + np.sqrt((more * more).mean(1, keepdims=True)) / m * np.abs(y)


def test_layer_as_a_graph():
    """Captured once, replayed with other inputs in place, eager calls of other sizes between the replays."""
    T = 33
    _, layer = make()
    _, eager = make()
    attention, residual = inputs(T)
    static_a, static_r = attention.clone(), residual.clone()
    codes, scales = outputs(T)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(static_a, static_r, codes, scales)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        layer(static_a, static_r, codes, scales)
    for rep in range(3):
        attention, residual = inputs(100 + rep)
        attention, residual = attention[:T], residual[:T].clone()
        static_a.copy_(attention)
        static_r.copy_(residual)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        c, s = eager(attention, residual, *outputs(T))
        assert torch.equal(residual, static_r) and torch.equal(c, codes) and torch.equal(s, scales), rep
        layer(*inputs(70 if rep else 5), *outputs(70 if rep else 5))  # a larger call may replace workspaces
        torch.cuda.synchronize()


@pytest.mark.parametrize("kind", ["bf16", "w8a8", "codes", "experts", "experts call"])
def test_capture_then_larger_calls(kind):
    """A captured call holds its workspaces when a larger call replaces them; split sums are in play."""
    N, Kk, small, large = 96, 4100, 5, (70, 900)
    c, s, _ = weights(3 * N, Kk, 1)
    if kind.startswith("experts"):
        s = np.stack([oracle.fp8b_quantize_ref(np.ones((N, Kk), np.float32), 128)[1]] * 3)
        h = sdg.SpenseExpertsFp8b(dev(c.reshape(3, N, Kk)), dev(s))
    else:
        h = sdg.SpenseLinearFp8b(dev(c), dev(s))
    offsets = {M: torch.tensor([0, M // 3, M // 3, M], dtype=torch.int32, device="cuda") for M in (small, *large)}

    def run(X, q, qs, Y):
        M = X.shape[0]
        if kind == "bf16":
            h(X, Y)
        elif kind == "w8a8":
            h.w8a8(X, Y)
        elif kind == "codes":
            h.quantized(q, qs, Y)
        elif kind == "experts":
            h.quantized(q, qs, offsets[M], Y)
        else:
            h(X, offsets[M], Y, adtype=sdg.DT_FP8)

    def case(M, yt):
        X, x = bf16(acts(M, Kk, M))
        q, qs = oracle.fp8b_quantize_ref(x)
        n = N if kind.startswith("experts") else 3 * N
        return X, dev(q), dev(qs), torch.full((M, n), float("nan"), dtype=yt, device="cuda")

    for yt in (torch.float32, torch.bfloat16):
        a = case(small, yt)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run(*a)
        torch.cuda.synchronize()
        want = a[3].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            run(*a)
        for M in large:
            b = case(M, yt)
            run(*b)
            torch.cuda.synchronize()
            assert not b[3].isnan().any()
            a[3].fill_(float("nan"))
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(a[3], want), (kind, M, yt)
        del g
    h.close()


def test_two_streams_at_once():
    """Handles of their own on two streams, and the calls that keep no state, do not meet."""
    c, s, _ = weights(300, 4096, 2)
    layers = [sdg.SpenseLinearFp8b(dev(c), dev(s)) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    X = [bf16(acts(20, 4096, i))[0] for i in range(2)]
    Y = [torch.empty((20, 300), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q = [(torch.empty((20, 4096), dtype=torch.uint8, device="cuda"), torch.empty((20, 32), device="cuda")) for _ in range(2)]
    want = []
    for i in range(2):
        layers[i].w8a8(X[i], Y[i])
        torch.cuda.synchronize()
        want.append(Y[i].clone())
        Y[i].zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                sdg.spense_block_norm(X[i], None, None, q[i][0], eps=1e-6, yscales=q[i][1])
                layers[i].w8a8(X[i], Y[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(Y[i], want[i])
        sc = torch.empty_like(q[i][0]), torch.empty_like(q[i][1])
        sdg.spense_block_norm(X[i], None, None, sc[0], eps=1e-6, yscales=sc[1])
        assert torch.equal(sc[0], q[i][0]) and torch.equal(sc[1], q[i][1])


def test_stream_argument():
    """The stream that is passed is the one that runs."""
    c, s, _ = weights(64, 256, 3)
    layer = sdg.SpenseLinearFp8b(dev(c), dev(s))
    X, _ = bf16(acts(8, 256, 4))
    Y, Z = torch.empty((8, 64), device="cuda"), torch.zeros((8, 64), device="cuda")
    layer(X, Y)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    layer(X, Z, stream=side)
    side.synchronize()
    assert torch.equal(Y, Z)


def test_example_runs(capsys, monkeypatch):
    monkeypatch.setattr("sys.argv", ["expert_block.py", "--tokens", "9", "--hidden", "256", "--intermediate", "64", "--experts", "4"])
    example.main()
    assert capsys.readouterr().out.count("us a call") == 3
