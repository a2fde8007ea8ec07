"""Cases of the microscaled 4-bit and expert operators, with their plain forms.

The operators: quantisation to microscaled 4-bit floating point (e2m1 values,
one power-of-two scale per 32 consecutive columns), the linear layer on such
weights, the linear layers of a set of experts over rows grouped by expert,
and the router that makes the groups.

Each case names its operator in ``op``.  ``run`` computes it in elementary
torch operations in 32 bits, or, with ``own`` set, through the package.
"""

from __future__ import annotations

import random

import torch

own = False

BLOCK = 32
H32, I32 = 5120, 25600      # hidden and intermediate size of the 32B-class FFN
I36, QKV36 = 27648, 12288   # intermediate size and QKV rows of the 36B-class layer
EXPERTS, IE = 16, 1600      # the 32B-class FFN cut into 16 experts


def listed():
    return [
        # the activations of one decoded token, ahead of a 4-bit projection: latency
        {"name": "quantize token", "op": "quantize", "M": 1, "K": H32, "x": "f32"},
        # the activations of a prefill step, ahead of the down projection
        {"name": "quantize prefill", "op": "quantize", "M": 2048, "K": I36, "x": "bf16"},
        # decode of one sequence: gate/up, bound by the weight bytes
        {"name": "linear decode 1", "op": "linear", "M": 1, "N": I32, "K": H32, "a": "bf16", "y": "bf16"},
        # decode of a batch: the long-K projection, partial sums kept in 32 bits
        {"name": "linear decode 32", "op": "linear", "M": 32, "N": H32, "K": I32, "a": "bf16", "y": "f32"},
        # prefill with activations left in bf16: QKV
        {"name": "linear prefill a16", "op": "linear", "M": 2048, "N": QKV36, "K": H32, "a": "bf16", "y": "bf16"},
        # a large decode batch with 4-bit activations: down
        {"name": "linear batch a4", "op": "linear", "M": 128, "N": H32, "K": I36, "a": "mx4", "y": "bf16"},
        # prefill with 4-bit activations: fused gate and up, the largest product
        {"name": "linear prefill a4", "op": "linear", "M": 2048, "N": 2 * I36, "K": H32, "a": "mx4", "y": "bf16"},
        # one decoded token through the router
        {"name": "route token", "op": "route", "T": 1, "E": EXPERTS, "k": 2, "l": "f32", "masked": False},
        # a ragged prefill through a router of many experts, some switched off for some tokens
        {"name": "route prefill", "op": "route", "T": 8191, "E": 128, "k": 8, "l": "bf16", "masked": True},
        # a decode batch through the experts' gate and up, 4-bit weights
        {"name": "experts decode", "op": "experts", "T": 13, "E": EXPERTS, "k": 2, "I": IE, "H": H32, "w": "mx4",
         "a": "bf16"},
        # prefill through the experts' gate and up, bf16 weights
        {"name": "experts prefill", "op": "experts", "T": 4096, "E": EXPERTS, "k": 2, "I": IE, "H": H32, "w": "bf16",
         "a": "bf16"},
        # prefill through the experts' down projection and the weighted sum over each token's experts, all 4-bit
        {"name": "experts down", "op": "down", "T": 2048, "E": EXPERTS, "k": 2, "I": IE, "H": H32, "w": "mx4",
         "a": "mx4"},
    ]


def _log(rng, lo, hi):
    v = int(round(lo * (hi / lo) ** rng.random()))
    return v + 1 if v == 3 * 1024 else v


def draw(rng: random.Random):
    op = rng.choice(["quantize", "linear", "linear", "route", "experts", "experts", "down"])
    if op == "quantize":
        M = _log(rng, 1, 8192)
        return {"op": op, "M": M, "K": _log(rng, 64, min(I36, 2048 * I36 // M)), "x": rng.choice(["f32", "bf16"])}
    if op == "linear":
        K = _log(rng, 96, I36)
        return {"op": op, "M": _log(rng, 1, 2048), "N": _log(rng, 64, min(2 * I36, 2 * I36 * H32 // K)), "K": K,
                "a": rng.choice(["bf16", "mx4"]), "y": rng.choice(["bf16", "f32"])}
    if op == "route":
        return {"op": op, "T": _log(rng, 1, 8192), "E": _log(rng, 8, 256), "k": rng.randint(1, 8),
                "l": rng.choice(["f32", "bf16"]), "masked": rng.random() < 0.5}
    E = _log(rng, 2, 64)
    return {"op": op, "T": _log(rng, 1, 4096), "E": E, "k": rng.randint(1, min(2, E)),
            "I": _log(rng, 64, min(3200, EXPERTS * IE // E)), "H": _log(rng, 128, H32),
            "w": rng.choice(["mx4", "bf16"]) if op == "experts" else "mx4",
            "a": "bf16" if op == "experts" else rng.choice(["bf16", "mx4"])}


# ---- the plain forms ----

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _blocks(x):
    """x [..., K] in 32 bits as [..., blocks, 32], the last block filled with zeros."""
    pad = -x.shape[-1] % BLOCK
    if pad:
        x = torch.cat([x, x.new_zeros(*x.shape[:-1], pad)], -1)
    return x.reshape(*x.shape[:-1], -1, BLOCK)


def _mx4(x):
    """Magnitude index (0..7), sign and exponent byte of every value of x [..., K]."""
    b = _blocks(x.float())
    amax = b.abs().amax(-1)
    e = (torch.frexp(amax)[1] + 124).clamp(0, 254)  # frexp: amax = f 2^e with f in [1/2, 1)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    q = torch.ldexp(b.abs(), 127 - e.unsqueeze(-1))
    code = ((q > 0.25).to(torch.uint8) + (q >= 0.75) + (q > 1.25) + (q >= 1.75) + (q > 2.5) + (q >= 3.5) + (q > 5.0))
    K = x.shape[-1]
    return code.flatten(-2)[..., :K], (b < 0).flatten(-2)[..., :K], e.to(torch.uint8)


def _values(code, neg, e, table):
    """The numbers that magnitude indexes, signs and exponent bytes stand for, in 32 bits."""
    v = table[code.int()]
    v = _blocks(torch.where(neg, -v, v))
    return torch.ldexp(v, e.unsqueeze(-1).int() - 127).flatten(-2)[..., : code.shape[-1]]


def _packed(code, neg):
    """Two codes in a byte, the even column in the low half."""
    c = code | (neg.to(torch.uint8) << 3)
    if c.shape[-1] % 2:
        c = torch.cat([c, c.new_zeros(*c.shape[:-1], 1)], -1)
    return c[..., ::2] | (c[..., 1::2] << 4)


def _weights(s):
    """The weights in 32 bits."""
    if s["w"] == "bf16":
        return s["W"].float()
    c = torch.stack([s["codes"] & 15, s["codes"] >> 4], -1).flatten(-2)[..., : s["K"]]
    return _values(c & 7, c >= 8, s["scales"], s["table"])


def _activations(s):
    return _values(*_mx4(s["X"]), s["table"]) if s["a"] == "mx4" else s["X"].float()


def _grouped(X, W, offsets, cap):
    """Rows of X [R, K], grouped by expert, through their expert's W [E, N, K]."""
    r = torch.arange(X.shape[0], device=X.device)
    e = (r[:, None] >= offsets[None, 1:]).sum(1)
    at = r - offsets.long()[e]
    P = X.new_zeros(W.shape[0], cap, X.shape[1])
    P[e, at] = X
    return torch.bmm(P, W.transpose(1, 2))[e, at]


def _route(logits, k, T, E):
    l = logits.float()
    l = torch.where(torch.isnan(l), torch.full_like(l, -float("inf")), l)
    v, i = torch.sort(l, dim=1, descending=True, stable=True)
    v, i = v[:, :k], i[:, :k]
    none = v == -float("inf")
    p = torch.where(none, torch.zeros_like(v), torch.exp(v - v[:, :1]))
    w = p / torch.where(none[:, :1], torch.ones_like(p[:, :1]), p.sum(1, keepdim=True))
    ids = torch.where(none, torch.full_like(i, -1), i).int()
    flat = torch.where(none, torch.full_like(i, E), i).flatten()
    order = torch.sort(flat, stable=True)[1]
    counts = (flat[:, None] == torch.arange(E, device=l.device)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    at = torch.arange(T * k, device=l.device)
    rows = torch.where(at < offsets[E], order // k, torch.full_like(order, -1)).int()
    pos = torch.empty_like(order)
    pos[order] = at
    pos = torch.where(none.flatten(), torch.full_like(pos, -1), pos).int().reshape(T, k)
    return {"ids": ids, "weights": w, "offsets": offsets, "rows": rows, "pos": pos}


# ---- inputs ----


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _acts(g, *shape):
    """Unit activations with one channel in 64 about eight times larger, as hidden states have them."""
    x = torch.randn(*shape, device="cuda", generator=g)
    big = torch.rand(shape[-1], device="cuda", generator=g) < 1 / 64
    return torch.where(big, 8 * x, x)


def _logits(g, T, E):
    """Router logits that make some experts much more popular than others."""
    return torch.randn(T, E, device="cuda", generator=g) + 0.8 * torch.randn(E, device="cuda", generator=g)


def prepare(case, seed):
    c = dict(case)
    g = _gen(seed)
    c["table"] = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")  # e2m1 magnitudes
    if c["op"] == "quantize":
        c["X"] = _acts(g, c["M"], c["K"]).to(_DT[c["x"]])
    elif c["op"] == "linear":
        c["w"] = "mx4"
        c["X"] = _acts(g, c["M"], c["K"]).bfloat16()
        code, neg, c["scales"] = _mx4(0.02 * torch.randn(c["N"], c["K"], device="cuda", generator=g))
        c["codes"] = _packed(code, neg)
    elif c["op"] == "route":
        c["logits"] = _logits(g, c["T"], c["E"]).to(_DT[c["l"]])
        if c["masked"]:
            off = torch.rand(c["T"], c["E"], device="cuda", generator=g) < 0.3
            c["logits"][off] = -float("inf")
    else:
        T, E, k = c["T"], c["E"], c["k"]
        r = _route(_logits(g, T, E), k, T, E)
        c["rows"], c["offsets"], c["pos"], c["weights"] = r["rows"], r["offsets"], r["pos"], r["weights"]
        c["cap"] = int((r["offsets"][1:] - r["offsets"][:-1]).max())
        up = c["op"] == "experts"
        N, c["K"] = (2 * c["I"], c["H"]) if up else (c["H"], c["I"])
        c["N"] = N
        c["X"] = _acts(g, T if up else T * k, c["K"]).bfloat16()
        W = 0.02 * torch.randn(E, N, c["K"], device="cuda", generator=g)
        if c["w"] == "mx4":
            code, neg, c["scales"] = _mx4(W)
            c["codes"] = _packed(code, neg)
        else:
            c["W"] = W.bfloat16()
    if own:
        _prepare_own(c)
    return c


def _empty(*shape, dtype):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def _prepare_own(c):
    """The packed weights, output buffers and workspace that a program keeps."""
    import sparse_dense_gemm_amd as sdg

    if c["op"] == "quantize":
        M, K = c["M"], c["K"]
        c["q"] = _empty(M, (K + 1) // 2, dtype=torch.uint8)
        c["e"] = _empty(M, -(-K // BLOCK), dtype=torch.uint8)
        c["Y"] = torch.empty_like(c["X"])
    elif c["op"] == "linear":
        c["layer"] = sdg.SpenseLinearMx4(c["codes"], c["scales"], K=c["K"])
        c["Y"] = _empty(c["M"], c["N"], dtype=_DT[c["y"]])
    elif c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        c["out"] = {"ids": _empty(T, k, dtype=torch.int32), "weights": _empty(T, k, dtype=torch.float32),
                    "offsets": _empty(E + 1, dtype=torch.int32), "rows": _empty(T * k, dtype=torch.int32),
                    "pos": _empty(T, k, dtype=torch.int32)}
        c["work"] = _empty(max(1, sdg.spense_route_workspace(T, E, k)), dtype=torch.uint8)
    else:
        if c["w"] == "mx4":
            c["layer"] = sdg.SpenseExperts(c["codes"], sdg.DT_MX4, scales=c["scales"], K=c["K"],
                                           glu=c["op"] == "experts")
        else:
            c["layer"] = sdg.SpenseExperts(c["W"], sdg.DT_BF16, glu=c["op"] == "experts")
        R = c["T"] * c["k"]
        if c["op"] == "experts":
            c["Y"] = _empty(R, c["I"], dtype=torch.bfloat16)
        else:
            c["O"] = _empty(R, c["H"], dtype=torch.float32)
            c["Y"] = _empty(c["T"], c["H"], dtype=torch.bfloat16)


# ---- one pass ----


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_plain(s):
    if s["op"] == "quantize":
        code, neg, e = _mx4(s["X"])
        return {"values": _values(code, neg, e, s["table"]).to(s["X"].dtype), "exponents": e}
    if s["op"] == "linear":
        return (_activations(s) @ _weights(s).T).to(_DT[s["y"]])
    if s["op"] == "route":
        return _route(s["logits"], s["k"], s["T"], s["E"])
    X = _activations(s)
    if s["op"] == "experts":
        gu = _grouped(X[s["rows"].long()], _weights(s), s["offsets"], s["cap"])
        gate, up = gu[:, : s["I"]], gu[:, s["I"]:]
        return (gate / (1 + torch.exp(-gate)) * up).bfloat16()
    O = _grouped(X, _weights(s), s["offsets"], s["cap"])
    return (O[s["pos"].long()] * s["weights"].unsqueeze(-1)).sum(1).bfloat16()


def _run_own(s):
    import sparse_dense_gemm_amd as sdg

    if s["op"] == "quantize":
        sdg.spense_quantize_mx4(s["X"], s["q"], s["e"])
        sdg.spense_dequantize_mx4(s["q"], s["e"], s["Y"])
        return {"values": s["Y"], "exponents": s["e"]}
    if s["op"] == "linear":
        return s["layer"].w4a4(s["X"], s["Y"]) if s["a"] == "mx4" else s["layer"](s["X"], s["Y"])
    if s["op"] == "route":
        o = s["out"]
        sdg.spense_route(s["logits"], s["k"], o["ids"], o["weights"], o["offsets"], o["rows"], o["pos"], s["work"])
        return o
    adtype = sdg.DT_MX4 if s["a"] == "mx4" else sdg.DT_BF16
    if s["op"] == "experts":
        return s["layer"](s["X"], s["offsets"], s["Y"], rows=s["rows"], adtype=adtype)
    s["layer"](s["X"], s["offsets"], s["O"], adtype=adtype)
    sdg.spense_experts_combine(s["O"], s["pos"], s["weights"], s["Y"])
    return s["Y"]


# ---- what a pass cannot do without ----


def work(case):
    c = case
    if c["op"] == "quantize":
        n, b = c["M"] * c["K"], {"f32": 4, "bf16": 2}[c["x"]]
        # the values in; codes and exponents out; the values they stand for out
        return {"bytes": n * (2 * b + 1 / 2 + 1 / BLOCK), "flops": 4 * n}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": N * K * (1 / 2 + 1 / BLOCK) + 2 * M * K + M * N * (4 if c["y"] == "f32" else 2),
                "flops": 2 * M * N * K}
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": T * E * (4 if c["l"] == "f32" else 2) + 16 * T * k + 4 * (E + 1), "flops": 4 * T * E}
    T, E, k, I, H = c["T"], c["E"], c["k"], c["I"], c["H"]
    R = T * k
    hit = E * (1 - (1 - k / E) ** T)  # experts that get a row, if all were as likely
    N, K = (2 * I, H) if c["op"] == "experts" else (H, I)
    weights = hit * N * K * (1 / 2 + 1 / BLOCK if c["w"] == "mx4" else 2)
    if c["op"] == "experts":
        return {"bytes": weights + 2 * T * H + 2 * R * I + 4 * R + 4 * E, "flops": 2 * R * N * K}
    return {"bytes": weights + 2 * R * I + 2 * T * H + 8 * R + 4 * E, "flops": 2 * R * N * K + 2 * R * H}


# ---- the same in 64 bits, from the definitions ----


def _e2m1(q):
    """The e2m1 number nearest to q >= 0, ties to the even one, nothing above 6."""
    step = 0.5 * (1 + (q >= 2) + 2 * (q >= 4).double())
    return (torch.round(q / step) * step).clamp(max=6.0)


def _exact_mx4(x):
    """The microscaled numbers nearest to x, and the powers of two they are multiples of."""
    x = x.double()
    K = x.shape[-1]
    x = torch.nn.functional.pad(x, (0, -K % BLOCK)).unflatten(-1, (-1, BLOCK))
    top = x.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(top > 0, top, torch.full_like(top, 2.0 ** -125)))) - 2
    e = e.clamp(-127, 127)
    return (torch.sign(x) * _e2m1(x.abs() * 2.0 ** -e) * 2.0 ** e).flatten(-2)[..., :K]


def _exact_weights(s):
    if s["w"] != "mx4":
        return s["W"].double()
    n = torch.stack([s["codes"] % 16, s["codes"] // 16], -1).flatten(-2)[..., : s["K"]].double()
    sign, n = 1 - 2 * (n >= 8).double(), n % 8
    exponent, fraction = torch.floor(n / 2), n % 2  # two exponent bits (bias 1), one fraction bit
    v = sign * torch.where(exponent == 0, fraction / 2, (1 + fraction / 2) * 2.0 ** (exponent - 1))
    return v * (2.0 ** (s["scales"].double() - 127)).repeat_interleave(BLOCK, -1)[..., : s["K"]]


def _exact_grouped(X, W, offsets):
    o = offsets.tolist()
    return torch.cat([X[o[e]:o[e + 1]] @ W[e].T for e in range(W.shape[0])])


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "quantize":
        return {"values": _exact_mx4(s["X"]), "exponents": None}
    if s["op"] == "route":
        l = torch.where(torch.isnan(s["logits"]), -float("inf"), s["logits"].double())
        v = l.topk(s["k"], 1)[0]
        e = torch.exp(v - v[:, :1])
        e = torch.where(torch.isnan(e), torch.zeros_like(e), e)
        total = e.sum(1, keepdim=True)
        return {"ids": None, "weights": e / torch.where(total > 0, total, torch.ones_like(total)), "offsets": None,
                "rows": None, "pos": None}
    X = _exact_mx4(s["X"]) if s["a"] == "mx4" else s["X"].double()
    W = _exact_weights(s)
    if s["op"] == "linear":
        return X @ W.T
    if s["op"] == "experts":
        gate, up = _exact_grouped(X[s["rows"].long()], W, s["offsets"]).chunk(2, -1)
        return gate * torch.sigmoid(gate) * up
    O = _exact_grouped(X, W, s["offsets"])
    return torch.einsum("tkn,tk->tn", O[s["pos"].long()], s["weights"].double())
