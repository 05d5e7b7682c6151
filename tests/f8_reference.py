"""The 8-bit floating point path in 64 bits, from its definition, and the bounds
that its kernels' results are held to.

Quantising, plain: a block's maximum is exact; f = 448 / max, v f and max / 448 are
single fp32 operations, and e4m3 of an fp32 number is exact to state.  So numbers
and scales are equal, bit for bit.  Gated by silu: v is off by e = (2 + |g|) 2u for
the exponential (counted twice) and 8 more roundings (u = 2^-24), so is max, and a
number q stands within half a step of some t' with |t' - t| <= (2 e + 4 u) |t|,
t = v 448 / max.

Projection: products of e4m3 numbers are exact (8 bits).  The sum of a block's 128
is off by at most 128 2^-23 of the sum of magnitudes (each addition by a unit in the
last place, should the tensor core cut off rather than round).  Scaling and adding
up the blocks takes 2 roundings a block and at most one addition for each block and
each CTA that shares K (8).  With S = sum |x||W|:
  |y - exact| <= (2^-16 + (nkb + 10) 2^-24) S + the output's rounding
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
BLOCK = 128
F8 = torch.float8_e4m3fn


def blocks(n: int) -> int:
    return -(-n // BLOCK)


def step(v):
    """Spacing of e4m3 numbers at |v| <= 448, in 64 bits."""
    exponent = ((v.double().view(torch.int64) >> 52) & 0x7FF).clamp(min=1023 - 6) - 3
    return (exponent << 52).view(torch.float64)


def e4m3(v):
    s = step(v)
    return torch.round(v.double() / s) * s


def quantised(v, tall=1):
    """(q as 64-bit values, scale fp32) of fp32 rows v [M, K], blocks of `tall` x 128: the stated fp32 operations."""
    assert v.dtype == torch.float32
    M, K = v.shape
    mb, kb = -(-M // tall), blocks(K)
    pad = torch.nn.functional.pad(v, (0, kb * BLOCK - K, 0, mb * tall - M)).view(mb, tall, kb, BLOCK)
    amax = pad.abs().amax(dim=(1, 3), keepdim=True)
    bad = ~pad.isfinite().all(dim=3, keepdim=True).all(dim=1, keepdim=True)
    up = torch.where(amax < 1e-30, 2.0 ** 100, 1.0).float()
    top = torch.full_like(amax, 448.0)       # a tensor: torch multiplies by the reciprocal of a number
    f = torch.where((amax > 0) & ~bad, top / (amax * up), torch.zeros_like(amax))
    prod = torch.where(f == 0, torch.zeros_like(pad), pad * up * f)
    scale = torch.where(bad, torch.full_like(amax, float("nan")), amax / top)
    q = e4m3(prod.clamp(-448, 448)).view(mb * tall, kb * BLOCK)[:M, :K]
    return q, scale.view(mb, kb)


def check_quantised(v, q, scale, tall=1):
    want_q, want_s = quantised(v.float(), tall)
    assert q.dtype is F8 and scale.dtype is torch.float32
    assert torch.equal(q.double(), want_q.to(q.device))
    assert bool(((scale == want_s) | (scale.isnan() & want_s.isnan())).all())


def check_gated(x, gate, q, scale):
    g, xd = gate.double(), x.double()
    v = xd * g / (1.0 + torch.exp(-g))
    e = ((2 + g.abs()) * 2 + 8) * U
    M, K = v.shape
    kb = blocks(K)

    def by_block(t):
        return torch.nn.functional.pad(t, (0, kb * BLOCK - K)).view(M, kb, BLOCK)

    amax, worst = by_block(v).abs().amax(2), by_block(e).amax(2)
    assert bool(((scale.double() - amax / 448).abs() <= (worst + 2 * U) * amax / 448 + 2.0 ** -150).all())
    wide = worst.repeat_interleave(BLOCK, 1)[:, :K]
    t = v * (448 / amax).repeat_interleave(BLOCK, 1)[:, :K]
    slack = (e + wide + 4 * U) * t.abs()
    high = (t.abs() + slack).clamp(max=448)
    assert bool(((q.double() - t).abs() <= step(high) / 2 + slack).all())


def values(q, scale, tall=1):
    s = scale.double().repeat_interleave(BLOCK, dim=-1)[..., :q.shape[-1]]
    if tall > 1:
        s = s.repeat_interleave(tall, dim=-2)[..., :q.shape[-2], :]
    return q.double() * s


def check_linear(x, xs, W, ws, residual, y, what=""):
    a, b = values(x, xs), values(W, ws, BLOCK)
    want, mass = a @ b.t(), a.abs() @ b.abs().t()
    tol = (2.0 ** -16 + (xs.shape[-1] + 10) * U) * mass
    if residual is not None:
        want = want + residual.double()
        tol = tol + U * want.abs()
    if y.dtype is torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs() + 2.0 ** -134
    off = (y.double() - want).abs() - tol
    assert bool((off <= 0).all()), f"{what}: off by {off.max().item()} beyond its bound at {off.argmax().item()}"
