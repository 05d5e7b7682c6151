"""The 8-bit path in 64 bits, from its definition, and the bounds that its
kernels' results are held to.

Rows.  With v the row in 64 bits and a = max|v|, t = v * 127 / a is what the
integer rounds.  The kernels work in fp32 (u = 2^-24): a sum of K squares, all
positive, whose longest chain of additions is at most K/64 + 24 long (at least
64 threads share a row, then a reduction), so mean(h^2) is off by at most
(K/64 + 24) u relatively, 1/sqrt by half of that, plus fewer than 16 roundings
(the sum h, the product with gamma, the quotient, the approximate exponential
counted as 2 + |g| units).  Call the total e.  Then
  |scale - a/127| <= e a/127,   |q - t| <= 1/2 + 127 * 2 e,   |y - v| <= (2^-8 + e)|v|.

Projection.  The integer sum is exact, and the four fp32 operations after it
are the same on both sides: results are equal, bit for bit.
"""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24


def row_error(K: int, gate=None) -> float:
    e = (0.5 * (K / 64 + 24) + 16) * U
    if gate is not None:
        e += (2 + float(gate.double().abs().max())) * 2 * U
    return e


def norm_rows(x, residual, gamma, eps):
    """(v, h) of the norm in 64 bits; CPU or GPU tensors."""
    h = x.double() if residual is None else x.double() + residual.double()
    v = h / torch.sqrt(h.square().mean(dim=1, keepdim=True) + eps)
    return (v if gamma is None else v * gamma.double()), h


def gated_rows(x, gate):
    v = x.double()
    if gate is not None:
        g = gate.double()
        v = v * g / (1.0 + torch.exp(-g))
    return v


def check_rows(v, q, scale, e: float, what: str = ""):
    """q, scale against the 64-bit rows v (all finite)."""
    a = v.abs().amax(dim=1)
    assert q.dtype == torch.int8 and scale.dtype == torch.float32
    zero = a == 0
    assert bool((q[zero] == 0).all()) and bool((scale[zero] == 0).all()), what
    live = ~zero
    v, a, q, scale = v[live], a[live], q[live].double(), scale[live].double()
    if not a.numel():
        return
    # scale may be subnormal: half its spacing, 2^-150, on top of the relative bound
    off = ((scale - a / 127).abs() - (e * a / 127 + 2.0 ** -150)).max().item()
    assert off <= 0, f"{what}: scale off by {off} beyond its bound"
    t = v * (127.0 / a)[:, None]
    worst = (q - t).abs().max().item()
    assert worst <= 0.5 + 127 * 2 * e, f"{what}: an integer is {worst} from its value"
    assert bool((q.abs().amax(dim=1) == 127).all()), f"{what}: a row's largest value is not 127"


def linear(x, x_scale, W, w_scale, residual, epilogue):
    """The projection's exact result: 64-bit integer-valued sums, then the
    four fp32 operations.  Returns what the kernel stores (bf16 or fp32)."""
    sums = x.double() @ W.double().t()                 # below 2^53: exact
    v = (sums.float() * x_scale[:, None]) * w_scale    # each operation rounded to fp32
    if residual is not None:
        v = v + residual.float()
    return v if epilogue == "fp32" else v.to(torch.bfloat16)


def same_bits(a, b):
    """Equal values, NaN in the same places."""
    return a.dtype == b.dtype and a.shape == b.shape and bool(((a == b) | (a.isnan() & b.isnan())).all())


def integers(g, rows, cols, lo=-127, hi=127):
    return torch.from_numpy(g.integers(lo, hi + 1, size=(rows, cols), dtype=np.int8))
