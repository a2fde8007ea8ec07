"""A decoder layer's expert block in microscaled 4-bit weights.

Each token goes through its k experts of E, every expert a GLU MLP:

    y[t] = sum_j weights[t, j] * down_e(silu(gate_e(x[t])) * up_e(x[t])),  e = ids[t, j]

in five launches on one stream and no synchronisation: the router (one or two),
gate and up of all experts at once, their down projections, and the weighted
sum.  Run it on an MI355X:

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
    block = ExpertBlock(*make(a.experts, a.hidden, a.intermediate), a.choices, a.tokens)
    X = torch.randn(a.tokens, a.hidden, device="cuda").bfloat16()
    Y = torch.empty_like(X)
    for name, adtype in (("bf16 activations", sdg.DT_BF16), ("mx4 activations", sdg.DT_MX4)):
        for _ in range(3):
            block(X, Y, adtype)
        start, end = torch.cuda.Event(True), torch.cuda.Event(True)
        start.record()
        for _ in range(20):
            block(X, Y, adtype)
        end.record()
        torch.cuda.synchronize()
        print(f"{a.tokens} tokens, {a.experts} experts, {a.choices} a token, {name}: "
              f"{start.elapsed_time(end) / 20 * 1e3:.1f} us a call, |Y| {Y.float().abs().mean():.3f}", flush=True)
    block.close()


if __name__ == "__main__":
    main()
