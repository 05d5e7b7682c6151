"""A gated MLP block in 8 bits: the operators of the 8-bit path as a decode or
prompt step uses them.

    h      = x + residual
    v      = rmsnorm(h) * gamma                        skg_rmsnorm_q8: h, 8-bit rows, and v in bf16
    u      = v . W_gate_up^T                           skg_q8_run
    a      = silu(u[:, :inner]) * u[:, inner:]         skg_quantize_q8: 8-bit rows
    out    = a . W_down^T + h                          skg_q8_run, residual in the epilogue
    scores = v . W_router^T                            skg_run (bf16 weights, fp32 scores), if there is a router

The weights are quantised once, one scale per output channel, by the same
quantiser.  A step allocates nothing and can be captured in a CUDA graph.

usage: python -m projection_gemm_gb300.q8_block [tokens] [hidden] [inner]
"""
from __future__ import annotations

import sys

import torch

from . import build, skg


def quantize_weight(W: torch.Tensor):
    """(int8 [N, K], fp32 [N]) of a bf16 weight [N, K] on the GPU."""
    q = torch.empty_like(W, dtype=torch.int8)
    scale = torch.empty(W.shape[0], dtype=torch.float32, device=W.device)
    skg.skg_quantize_q8(W, None, q, scale)
    return q, scale


class Q8MLP:
    """Plans, 8-bit weights and buffers of one block for M tokens."""

    def __init__(self, M: int, gamma, W_gate_up, W_down, W_router=None, eps: float = 1e-6):
        hidden, inner = W_down.shape
        if W_gate_up.shape != (2 * inner, hidden) or gamma.shape != (hidden,):
            raise ValueError("W_gate_up is [2 inner, hidden], W_down [hidden, inner], gamma [hidden]")
        self.M, self.hidden, self.inner, self.eps, self.gamma = M, hidden, inner, eps, gamma
        self.gate_up, self.gate_up_scale = quantize_weight(W_gate_up)
        self.down, self.down_scale = quantize_weight(W_down)
        # from here on the weights are static: the plans may fetch them early
        torch.cuda.current_stream().synchronize()
        self.p_up = skg.Q8Plan(M, 2 * inner, hidden, "bf16", static_weights=True)
        self.p_down = skg.Q8Plan(M, hidden, inner, "bf16_residual", static_weights=True)
        dev = W_down.device
        self.h = torch.empty(M, hidden, dtype=torch.bfloat16, device=dev)
        self.q = torch.empty(M, hidden, dtype=torch.int8, device=dev)
        self.scale = torch.empty(M, dtype=torch.float32, device=dev)
        self.u = torch.empty(M, 2 * inner, dtype=torch.bfloat16, device=dev)
        self.a = torch.empty(M, inner, dtype=torch.int8, device=dev)
        self.a_scale = torch.empty(M, dtype=torch.float32, device=dev)
        self.out = torch.empty(M, hidden, dtype=torch.bfloat16, device=dev)
        self.W_router = W_router
        self.v = self.scores = self.p_router = None
        if W_router is not None:
            self.p_router = skg.Plan(M, W_router.shape[0], hidden, "fp32")      # M <= 64
            self.v = torch.empty(M, hidden, dtype=torch.bfloat16, device=dev)
            self.scores = torch.empty(M, W_router.shape[0], dtype=torch.float32, device=dev)

    def run(self, x, residual, stream=None):
        """One step; x, residual bf16 [M, hidden].  Returns (out, scores or None), buffers of this block."""
        skg.skg_rmsnorm_q8(x, residual, self.gamma, self.eps, self.h, self.q, self.scale, self.v, stream)
        self.p_up.run(self.q, self.scale, self.gate_up, self.gate_up_scale, None, self.u, stream)
        skg.skg_quantize_q8(self.u[:, self.inner:], self.u[:, :self.inner], self.a, self.a_scale, stream)
        self.p_down.run(self.a, self.a_scale, self.down, self.down_scale, self.h, self.out, stream)
        if self.p_router is not None:
            # Last, although v is there since the norm: between the norm and the up projection it keeps the
            # latter's early CTAs off its SMs.  One token, 7168 x 8192: 66.6 us there, 40.9 us here; 64: 68.3, 66.2.
            self.p_router.run(self.v, self.W_router, None, self.scores, stream)
        return self.out, self.scores

    def check(self):
        for p in (self.p_up, self.p_down, self.p_router):
            if p is not None:
                p.check()

    def close(self):
        for p in (self.p_up, self.p_down, self.p_router):
            if p is not None:
                p.close()


def main(argv):
    M, hidden, inner = (int(v) for v in (list(argv) + ["16", "7168", "8192"][len(argv):]))
    build.build()
    skg.load()
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)

    gamma, x, r = normal(hidden, std=0.1) + 1, normal(M, hidden), normal(M, hidden)
    W1, W2 = normal(2 * inner, hidden, std=hidden ** -0.5), normal(hidden, inner, std=inner ** -0.5)
    block = Q8MLP(M, gamma, W1, W2, normal(384, hidden, std=hidden ** -0.5) if M <= 64 else None)
    out, _ = block.run(x, r)
    block.check()

    h = x.float() + r.float()
    v = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + 1e-6) * gamma.float()
    u = v @ W1.float().t()
    want = (torch.nn.functional.silu(u[:, :inner]) * u[:, inner:]) @ W2.float().t()
    got = out.float() - h
    print(f"M={M} hidden={hidden} inner={inner}: the block's contribution is "
          f"{((got - want).norm() / want.norm()).item():.3%} off the unquantised one")

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.run(x, r)
    steps, times = 50, []
    for _ in range(10):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(steps):
            graph.replay()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b) * 1e3 / steps)
    block.check()
    weights = block.gate_up.numel() + block.down.numel()
    us = sorted(times)[len(times) // 2]
    print(f"one step as a CUDA graph, back to back: {us:.1f} us, {weights / us / 1e3:.0f} GB/s of 8-bit weights")
    block.close()


if __name__ == "__main__":
    main(sys.argv[1:])
