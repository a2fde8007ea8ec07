"""A decoder layer's expert block in microscaled 4-bit weights, and one between
its two norms in block-scaled 8 bits.

Each token goes through its k experts of E, every expert a GLU MLP:

    y[t] = sum_j weights[t, j] * down_e(silu(gate_e(x[t])) * up_e(x[t])),  e = ids[t, j]

in five launches on one stream and no synchronisation: the router (one or two),
gate and up of all experts at once, their down projections, and the weighted
sum.  In 8 bits (ExpertLayer8) the passes around the block belong to it: the
residual takes the output of the block before, its norm goes out in 8 bits for
the router and the experts, and the residual takes the experts' weighted sum with
the next norm.  Run it on an MI355X:

    python examples/expert_block.py [--tokens 256] [--hidden 5120] [--intermediate 1600] [--experts 16] [--choices 2]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import sparse_dense_gemm_amd as sdg  # noqa: E402


def quantized(W):
    """Codes and exponent bytes of weights [E, N, K]."""
    E, N, K = W.shape
    codes = torch.empty((E, N, (K + 1) // 2), dtype=torch.uint8, device=W.device)
    scales = torch.empty((E, N, (K + 31) // 32), dtype=torch.uint8, device=W.device)
    sdg.spense_quantize_mx4(W.view(E * N, K), codes.view(E * N, -1), scales.view(E * N, -1))
    return codes, scales


class ExpertBlock:
    """gate_up [E, 2I, H] (rows [0, I) the gate), down [E, H, I], router [E, H]; for up to max_tokens tokens a call."""

    def __init__(self, gate_up, down, router, choices: int, max_tokens: int):
        E, I2, H = gate_up.shape
        self.k, self.router = choices, router.bfloat16()
        codes, scales = quantized(gate_up)
        self.gate_up = sdg.SpenseExperts(codes, sdg.DT_MX4, scales=scales, K=H, glu=True)
        codes, scales = quantized(down)
        self.down = sdg.SpenseExperts(codes, sdg.DT_MX4, scales=scales, K=I2 // 2)
        R = max_tokens * choices
        i32 = dict(dtype=torch.int32, device=gate_up.device)
        self.ids, self.pos = torch.empty((max_tokens, choices), **i32), torch.empty((max_tokens, choices), **i32)
        self.weights = torch.empty((max_tokens, choices), device=gate_up.device)
        self.offsets, self.rows = torch.empty(E + 1, **i32), torch.empty(R, **i32)
        need = sdg.spense_route_workspace(max_tokens, E, choices)
        self.work = torch.empty(max(1, need), dtype=torch.uint8, device=gate_up.device)
        self.A = torch.empty((R, I2 // 2), dtype=torch.bfloat16, device=gate_up.device)
        self.O = torch.empty((R, H), device=gate_up.device)

    def __call__(self, X, Y, adtype: int = sdg.DT_BF16):
        """Y[t] of X [T, H] bf16; adtype sdg.DT_MX4 quantises the activations ahead of both projections."""
        T = X.shape[0]
        R = T * self.k
        logits = X @ self.router.T
        ids, pos, weights = self.ids[:T], self.pos[:T], self.weights[:T]
        sdg.spense_route(logits, self.k, ids, weights, self.offsets, self.rows, pos, self.work)
        self.gate_up(X, self.offsets, self.A[:R], rows=self.rows, adtype=adtype)
        self.down(self.A[:R], self.offsets, self.O[:R], adtype=adtype)
        sdg.spense_experts_combine(self.O[:R], pos, weights, Y)
        return Y

    def close(self):
        self.gate_up.close()
        self.down.close()


def quantized8(W):
    """Codes and block scales of weights [N, K]."""
    N, K = W.shape
    codes = torch.empty((N, K), dtype=torch.uint8, device=W.device)
    scales = torch.empty((-(-N // 128), -(-K // 128)), device=W.device)
    sdg.spense_quantize_fp8b(W.contiguous(), codes, scales, rows=128)
    return codes, scales


def quantized8_experts(W, parts=1):
    """The same of experts' weights [E, N, K], `parts` matrices of equal height to an expert."""
    each = [quantized8(p) for w in W for p in w.chunk(parts)]
    codes, scales = (torch.stack(t) for t in zip(*each))
    return codes.view(W.shape), scales.view(W.shape[0], -1, scales.shape[-1])


class ExpertLayer8:
    """An expert block between two norms, weights and activations in block-scaled 8 bits:

        residual += rms(attention) * post                  codes = fp8b(rms(residual) * pre)
        residual += gate * sum_j weights[:, j] expert_(ids[:, j])(codes)
        next = fp8b(rms(residual) * pre_next)

    gate_up [E, 2I, H] (rows [0, I) the gate), down [E, H, I], router [E, H]; post, pre, gate, pre_next [H]; for up to
    max_tokens tokens a call."""

    def __init__(self, gate_up, down, router, norms, choices: int, max_tokens: int, eps: float = 1e-6):
        E, I2, H = gate_up.shape
        self.k, self.E, self.norms, self.eps = choices, E, norms, eps
        self.gate_up = sdg.SpenseExpertsFp8b(*quantized8_experts(gate_up, 2), glu=True)
        self.down = sdg.SpenseExpertsFp8b(*quantized8_experts(down))
        self.router = sdg.SpenseLinearFp8b(*quantized8(router))
        R = max_tokens * choices
        d = gate_up.device
        i32, u8 = dict(dtype=torch.int32, device=d), dict(dtype=torch.uint8, device=d)
        self.codes, self.scales = torch.empty((max_tokens, H), **u8), torch.empty((max_tokens, -(-H // 128)), device=d)
        self.logits = torch.empty((max_tokens, E), device=d)
        self.ids, self.pos = torch.empty((max_tokens, choices), **i32), torch.empty((max_tokens, choices), **i32)
        self.weights = torch.empty((max_tokens, choices), device=d)
        self.offsets, self.rows = torch.empty(E + 1, **i32), torch.empty(R, **i32)
        self.work = torch.empty(max(1, sdg.spense_route_workspace(max_tokens, E, choices)), **u8)
        self.A = torch.empty((R, I2 // 2), dtype=torch.bfloat16, device=d)
        self.O = torch.empty((R, H), device=d)

    def __call__(self, attention, residual, codes, scales):
        """attention, residual [T, H] bf16, the residual updated in place; codes and scales: the next block's activations."""
        T = attention.shape[0]
        R, n = T * self.k, self.norms
        c, s, logits = self.codes[:T], self.scales[:T], self.logits[:T]
        ids, pos, weights = self.ids[:T], self.pos[:T], self.weights[:T]
        sdg.spense_block_norm(attention, residual, residual, c, post=n["post"], pre=n["pre"], eps=self.eps, yscales=s)
        self.router.quantized(c, s, logits)
        sdg.spense_route(logits, self.k, ids, weights, self.offsets, self.rows, pos, self.work)
        self.gate_up.quantized(c, s, self.offsets, self.A[:R], rows=self.rows)
        self.down(self.A[:R], self.offsets, self.O[:R], adtype=sdg.DT_FP8)
        sdg.spense_block_norm(self.O[:R], residual, residual, codes, pre=n["pre_next"], gate=n["gate"], eps=self.eps,
                              yscales=scales, pos=pos, weights=weights)
        return codes, scales

    def close(self):
        for layer in (self.gate_up, self.down, self.router):
            layer.close()


def make_norms(H, device="cuda", seed=1):
    g = torch.Generator(device=device).manual_seed(seed)
    n = {k: (1 + 0.2 * torch.randn(H, device=device, generator=g)).bfloat16() for k in ("post", "pre", "pre_next")}
    n["gate"] = torch.tanh(torch.randn(H, device=device, generator=g)).bfloat16()
    return n


def make(E, H, I, device="cuda", seed=0):
    g = torch.Generator(device=device).manual_seed(seed)
    gate_up = torch.randn(E, 2 * I, H, device=device, generator=g) / H ** 0.5
    down = torch.randn(E, H, I, device=device, generator=g) / I ** 0.5
    router = torch.randn(E, H, device=device, generator=g) / H ** 0.5
    return gate_up, down, router


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=256)
    ap.add_argument("--hidden", type=int, default=5120)
    ap.add_argument("--intermediate", type=int, default=1600)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--choices", type=int, default=2)
    a = ap.parse_args()
    weights = make(a.experts, a.hidden, a.intermediate)
    block = ExpertBlock(*weights, a.choices, a.tokens)
    layer = ExpertLayer8(*weights, make_norms(a.hidden), a.choices, a.tokens)
    X = torch.randn(a.tokens, a.hidden, device="cuda").bfloat16()
    Y = torch.empty_like(X)
    codes, scales = torch.empty_like(layer.codes), torch.empty_like(layer.scales)
    for name, call in (("mx4 weights, bf16 activations", lambda: block(X, Y, sdg.DT_BF16)),
                       ("mx4 weights and activations", lambda: block(X, Y, sdg.DT_MX4)),
                       ("8 bits with both norms", lambda: layer(X, Y, codes, scales))):
        for _ in range(3):
            call()
        start, end = torch.cuda.Event(True), torch.cuda.Event(True)
        start.record()
        for _ in range(20):
            call()
        end.record()
        torch.cuda.synchronize()
        print(f"{a.tokens} tokens, {a.experts} experts, {a.choices} a token, {name}: "
              f"{start.elapsed_time(end) / 20 * 1e3:.1f} us a call, |Y| {Y.float().abs().mean():.3f}", flush=True)
    block.close()
    layer.close()


if __name__ == "__main__":
    main()
