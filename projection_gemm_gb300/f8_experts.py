"""A layer of experts in 8-bit floating point: the operators of that path as a
decode or prompt step uses them.

    scores = x . W_router^T                            skg_run (bf16 weights, fp32 scores), up to 64 tokens
    expert, weight = the k best of softmax(scores)     (torch)
    offsets, rows, pos                                 skg_experts_sort: the T * k choices by expert
    q      = x[rows] in blocks of 128                  skg_quantize_f8
    u      = q . W_gate_up[expert]^T                   skg_f8_run with experts
    a      = silu(u[:, :inner]) * u[:, inner:]         skg_quantize_f8
    d      = a . W_down[expert]^T                      skg_f8_run with experts
    out[t] = residual[t] + sum_j weight[t,j] d[pos[t,j]]      skg_experts_combine

The weights are quantised once, a scale for each block of 128 x 128.  A step from
given choices allocates nothing and can be captured in a CUDA graph.

usage: python -m projection_gemm_gb300.f8_experts [tokens] [hidden] [inner] [experts] [k]
"""
from __future__ import annotations

import contextlib
import sys

import torch

from . import build, skg


def quantize_weights(W: torch.Tensor):
    """(float8_e4m3fn, fp32 scales) of bf16 weights [experts, N, K] on the GPU."""
    E, N, K = W.shape
    q = torch.empty_like(W, dtype=torch.float8_e4m3fn)
    scale = torch.empty(E, -(-N // 128), -(-K // 128), dtype=torch.float32, device=W.device)
    skg.skg_quantize_f8_weights(W, q, scale)
    return q, scale


def on_stream(stream):
    """torch's operators on the stream that the library's calls are given: a stream, its handle, or None for the current."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


class F8Experts:
    """Plans, 8-bit weights and buffers of one layer for T tokens that choose k experts each."""

    def __init__(self, T: int, k: int, W_gate_up, W_down, W_router=None):
        E, hidden, inner = W_down.shape
        if W_gate_up.shape != (E, 2 * inner, hidden):
            raise ValueError("W_gate_up is [experts, 2 inner, hidden], W_down [experts, hidden, inner]")
        self.T, self.k, self.E, self.hidden, self.inner = T, k, E, hidden, inner
        self.gate_up, self.gate_up_scale = quantize_weights(W_gate_up)
        self.down, self.down_scale = quantize_weights(W_down)
        R, dev = T * k, W_down.device
        self.p_up = skg.F8Plan(R, 2 * inner, hidden, "bf16", experts=E, static_weights=True)
        self.p_down = skg.F8Plan(R, hidden, inner, "bf16", experts=E, static_weights=True)

        def empty(*shape, dtype=torch.bfloat16):
            return torch.empty(*shape, dtype=dtype, device=dev)

        self.offsets = empty(E + 1, dtype=torch.int32)
        self.rows, self.pos = empty(R, dtype=torch.int32), empty(T, k, dtype=torch.int32)
        self.q, self.q_scale = empty(R, hidden, dtype=torch.float8_e4m3fn), empty(R, -(-hidden // 128), dtype=torch.float32)
        # rows of no expert are never written, and never read: zeros, so that nothing is made of chance bits
        self.u, self.d = torch.zeros(R, 2 * inner, dtype=torch.bfloat16, device=dev), empty(R, hidden)
        self.a, self.a_scale = empty(R, inner, dtype=torch.float8_e4m3fn), empty(R, -(-inner // 128), dtype=torch.float32)
        self.out = empty(T, hidden)
        self.W_router, self.p_router = W_router, None
        if W_router is not None:
            self.p_router = skg.Plan(T, E, hidden, "fp32")      # T <= 64
            self.scores = empty(T, E, dtype=torch.float32)
        # from here on the weights are static, and the zeros there for a step on any stream
        torch.cuda.current_stream().synchronize()

    def route(self, x, stream=None):
        """(expert int32, weight fp32) [T, k]: the k best experts of each token by the router's softmax."""
        self.p_router.run(x, self.W_router, None, self.scores, stream)
        with on_stream(stream):
            weight, expert = torch.topk(torch.softmax(self.scores, dim=1), self.k, dim=1)
            return expert.to(torch.int32), weight

    def run(self, x, residual, expert, weight, stream=None):
        """One step; x, residual bf16 [T, hidden] (residual may be None), expert int32 and weight fp32 [T, k].  Returns
        out, a buffer of this layer."""
        skg.skg_experts_sort(expert, self.offsets, self.rows, self.pos, stream)
        skg.skg_quantize_f8(x, None, self.q, self.q_scale, rows=self.rows, stream=stream)
        self.p_up.run(self.q, self.q_scale, self.gate_up, self.gate_up_scale, None, self.u, offsets=self.offsets, stream=stream)
        skg.skg_quantize_f8(self.u[:, self.inner:], self.u[:, :self.inner], self.a, self.a_scale, stream=stream)
        self.p_down.run(self.a, self.a_scale, self.down, self.down_scale, None, self.d, offsets=self.offsets, stream=stream)
        skg.skg_experts_combine(self.d, self.pos, weight, residual, self.out, stream)
        return self.out

    def check(self):
        for p in (self.p_up, self.p_down, self.p_router):
            if p is not None:
                p.check()

    def close(self):
        for p in (self.p_up, self.p_down, self.p_router):
            if p is not None:
                p.close()


def main(argv):
    T, hidden, inner, E, k = (int(v) for v in (list(argv) + ["16", "4096", "1024", "64", "8"][len(argv):]))
    build.build()
    skg.load()
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)

    x, r = normal(T, hidden), normal(T, hidden)
    W1, W2 = normal(E, 2 * inner, hidden, std=hidden ** -0.5), normal(E, hidden, inner, std=inner ** -0.5)
    W_router = normal(E, hidden, std=hidden ** -0.5)
    layer = F8Experts(T, k, W1, W2, W_router if T <= 64 else None)
    if T <= 64:
        expert, weight = layer.route(x)
    else:
        weight, expert = torch.topk(torch.softmax(x.float() @ W_router.float().t(), dim=1), k, dim=1)
        expert = expert.to(torch.int32)
    out = layer.run(x, r, expert, weight)
    layer.check()

    want = torch.zeros(T, hidden, device="cuda")
    for e in range(E):
        t, j = (expert == e).nonzero(as_tuple=True)
        u = x[t].float() @ W1[e].float().t()
        v = (torch.nn.functional.silu(u[:, :inner]) * u[:, inner:]) @ W2[e].float().t()
        want.index_add_(0, t, v * weight[t, j, None])
    got = out.float() - r.float()
    print(f"T={T} hidden={hidden} inner={inner} experts={E} k={k}: the layer's contribution is "
          f"{((got - want).norm() / want.norm()).item():.3%} off the unquantised one")

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.run(x, r, expert, weight)
    steps, times = 50, []
    for _ in range(10):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(steps):
            graph.replay()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b) * 1e3 / steps)
    layer.check()
    taken = len(torch.unique(expert))
    us = sorted(times)[len(times) // 2]
    print(f"one step as a CUDA graph, back to back: {us:.1f} us, {taken} experts, "
          f"{taken * 3 * inner * hidden / us / 1e3:.0f} GB/s of their 8-bit weights")
    layer.close()


if __name__ == "__main__":
    main(sys.argv[1:])
