"""The 8-bit projection path as measured cases: the norm and the quantiser that write 8-bit activations, and
the 8-bit projection that reads them.

Each case is one operator at one size.  ``run`` computes it either in plain torch operations (32-bit
arithmetic, one rounding at the end) or, where ``own`` is true, with this library's entry points; ``exact``
computes it in 64 bits, from the definition:

  norm    h = x + residual;  y = h / sqrt(mean(h^2) + eps) * gamma;  (q, scale) = rows(y)
  quant   v = x, or silu(gate) * x;                                  (q, scale) = rows(v)
  linear  y[m, n] = x_scale[m] * w_scale[n] * sum_k x[m, k] W[n, k]  (+ residual[m, n])

  rows(y): scale = max|y| / 127 of each row, q = y * 127 / max|y| rounded to the nearest integer (half to even)

Rows held in 8 bits are returned as the values they stand for, q * scale, in the activations' own type (bf16).
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6


def listed():
    return [
        # one decode token entering a layer of the 7168-wide model of this library's decode chain
        {"name": "norm m1", "op": "norm", "M": 1, "K": 7168, "residual": True},
        # the largest decode batch
        {"name": "norm m64", "op": "norm", "M": 64, "K": 7168, "residual": True},
        # a prompt of 8192 tokens, where the norm streams through HBM
        {"name": "norm m8192", "op": "norm", "M": 8192, "K": 7168, "residual": True},
        # a gated activation between two projections at a decode batch
        {"name": "gate m16", "op": "quant", "M": 16, "K": 16384, "gated": True},
        # rows of odd length (nothing is 16-byte aligned): an attention output with a ragged width
        {"name": "quant m1023 odd", "op": "quant", "M": 1023, "K": 5001, "gated": False},
        # the gated activation of a long prompt
        {"name": "gate m4096", "op": "quant", "M": 4096, "K": 16384, "gated": True},
        # the smallest projection here (1024 x 1024, one token): latency alone
        {"name": "linear m1 1024", "op": "linear", "M": 1, "N": 1024, "K": 1024, "epilogue": "bf16_residual"},
        # one token through the wide input projection
        {"name": "linear m1 wide", "op": "linear", "M": 1, "N": 12288, "K": 7168, "epilogue": "bf16"},
        # the middle of the batch sweep
        {"name": "linear m16", "op": "linear", "M": 16, "N": 7168, "K": 7168, "epilogue": "bf16"},
        # the largest decode batch through the deep-K output projection, residual added
        {"name": "linear m64 deep", "op": "linear", "M": 64, "N": 7168, "K": 16384, "epilogue": "bf16_residual"},
        # a short prompt with ragged sizes, scores kept in fp32
        {"name": "linear m333 odd", "op": "linear", "M": 333, "N": 5001, "K": 4112, "epilogue": "fp32"},
        # a long prompt through the wide input projection
        {"name": "linear m4096 wide", "op": "linear", "M": 4096, "N": 12288, "K": 7168, "epilogue": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "quant", "linear", "linear"])
    if op == "norm":
        K = _log(rng, 256, 16384)
        return {"op": op, "M": _log(rng, 1, min(8192, 8192 * 7168 // K)), "K": K, "residual": rng.random() < 0.75}
    if op == "quant":
        return {"op": op, "M": _log(rng, 1, 4096), "K": _log(rng, 256, 16384), "gated": rng.random() < 0.5}
    N, K = _log(rng, 64, 16384), 16 * _log(rng, 16, 1024)
    M = _log(rng, 1, max(1, min(4096, 4096 * 12288 * 7168 // (N * K))))
    return {"op": op, "M": M, "N": N, "K": K, "epilogue": rng.choice(["bf16", "bf16_residual", "fp32"])}


# ------------------------------------------------------------------------------------------------ inputs
def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    def integers(rows, cols):     # quantised normal rows: the largest of a few thousand is about 4 sigma = 127
        v = torch.randn(rows, cols, generator=g, device="cuda")
        return v.mul_(32.0).round_().clamp_(-127, 127).to(torch.int8)

    def positive(n, mean):
        return mean * (0.5 + torch.rand(n, generator=g, device="cuda"))

    s = {"op": case["op"], "M": case["M"], "K": case["K"]}
    M, K = case["M"], case["K"]
    if case["op"] == "norm":
        s["x"] = normal(M, K)
        s["residual"] = normal(M, K, std=2.0) if case["residual"] else None
        s["gamma"] = (1.0 + 0.25 * torch.randn(K, generator=g, device="cuda")).to(torch.bfloat16)
        s["gamma"][torch.randint(K, (max(1, K // 200),), generator=g, device="cuda")] *= 4   # outlier channels
    elif case["op"] == "quant":
        # one [M, 2K] output of a fused gate/up projection: both halves are strided views of it
        both = normal(M, 2 * K if case["gated"] else K, std=1.5)
        s["gate"] = both[:, :K] if case["gated"] else None
        s["x"] = both[:, K:] if case["gated"] else both
    else:
        N = case["N"]
        s["N"], s["epilogue"] = N, case["epilogue"]
        s["x"], s["x_scale"] = integers(M, K), positive(M, 1.0 / 32)
        s["W"], s["w_scale"] = integers(N, K), positive(N, 1.0 / (32 * math.sqrt(K)))
        s["residual"] = normal(M, N) if case["epilogue"] == "bf16_residual" else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:      # the plan and the buffers that a program keeps
        from projection_gemm_gb300 import skg
        M, K = case["M"], case["K"]
        if case["op"] == "linear":
            s["plan"] = skg.Q8Plan(M, s["N"], K, s["epilogue"], static_weights=True)
            s["y"] = torch.empty(M, s["N"], device="cuda",
                                 dtype=torch.float32 if s["epilogue"] == "fp32" else torch.bfloat16)
        else:
            s["q"] = torch.empty(M, K, dtype=torch.int8, device="cuda")
            s["scale"] = torch.empty(M, dtype=torch.float32, device="cuda")
            s["values"] = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
            if case["op"] == "norm":
                s["h"] = torch.empty_like(s["x"]) if s["residual"] is not None else None
    return s


# ------------------------------------------------------------------------------------------- plain form
def _rows(y):
    largest = y.abs().amax(dim=1, keepdim=True)
    q = torch.round(y * (127.0 / largest))
    scale = largest / 127.0
    return (q * scale).to(torch.bfloat16), scale[:, 0]


def _plain(s):
    if s["op"] == "norm":
        h = s["x"].float()
        if s["residual"] is not None:
            h = h + s["residual"].float()
        y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS) * s["gamma"].float()
        values, scale = _rows(y)
        return {"values": values, "scale": scale,
                "h": h.to(torch.bfloat16) if s["residual"] is not None else None}
    if s["op"] == "quant":
        v = s["x"].float()
        if s["gate"] is not None:
            g = s["gate"].float()
            v = g / (1.0 + torch.exp(-g)) * v
        values, scale = _rows(v)
        return {"values": values, "scale": scale}
    y = (s["x"].float() @ s["W"].float().t()) * s["x_scale"][:, None] * s["w_scale"]
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y if s["epilogue"] == "fp32" else y.to(torch.bfloat16)}


# ------------------------------------------------------------------------------------ this library's form
def _own(s):
    from projection_gemm_gb300 import skg
    if s["op"] == "linear":
        s["plan"].run(s["x"], s["x_scale"], s["W"], s["w_scale"], s["residual"], s["y"])
        return {"y": s["y"]}
    if s["op"] == "norm":
        skg.skg_rmsnorm_q8(s["x"], s["residual"], s["gamma"], EPS, s["h"], s["q"], s["scale"])
    else:
        skg.skg_quantize_q8(s["x"], s["gate"], s["q"], s["scale"])
    torch.mul(s["q"], s["scale"][:, None], out=s["values"])
    return {"values": s["values"], "scale": s["scale"], **({"h": s["h"]} if s["op"] == "norm" else {})}


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------------------------- 64-bit values
def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "linear":
        sums = torch.mm(s["x"].double(), s["W"].double().T)      # integers below 2^53: no rounding
        y = torch.outer(s["x_scale"].double(), s["w_scale"].double()) * sums
        return {"y": y if s["residual"] is None else y + s["residual"].double()}
    v, h = s["x"].double(), None
    if case["op"] == "norm":
        if s["residual"] is not None:
            v = h = v + s["residual"].double()
        v = v / torch.sqrt(v.square().sum(1, keepdim=True) / case["K"] + EPS) * s["gamma"].double()
    elif s["gate"] is not None:
        g = s["gate"].double()
        v = torch.sigmoid(g) * g * v
    step = v.abs().max(1, keepdim=True).values / 127
    answer = {"values": torch.round(v / step) * step, "scale": step.squeeze(1)}
    return {**answer, "h": h} if case["op"] == "norm" else answer


# ------------------------------------------------------------------------------------------------- work
def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "norm":
        streams = 3 if case["residual"] else 1                  # x, and with a residual it and h, in bf16
        return {"bytes": 2 * streams * M * K + M * K + 2 * K + 4 * M, "flops": 7 * M * K}
    if case["op"] == "quant":
        streams = 2 if case["gated"] else 1
        return {"bytes": 2 * streams * M * K + M * K + 4 * M, "flops": (8 if case["gated"] else 3) * M * K}
    N = case["N"]
    out = {"bf16": 2, "bf16_residual": 4, "fp32": 4}[case["epilogue"]]
    return {"bytes": N * K + M * K + 4 * (M + N) + out * M * N, "flops": 2 * M * N * K}
