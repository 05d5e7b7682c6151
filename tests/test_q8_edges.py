"""The 8-bit path where a bound leaves room: integers that have to be equal,
values at the ends of their types' ranges, and sizes at the ends of theirs."""
import numpy as np
import pytest
import torch

from projection_gemm_gb300 import skg
from tests import q8_reference as R
from tests.test_q8_gpu import normal, rng, rows_out


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from projection_gemm_gb300 import build
    build.build()
    skg.load()


def nearest_even(v):
    """127 v / max|v| of each row rounded to the nearest integer, half to even, in integers: bf16 values are
    8-bit integers times powers of two, so twice the quotient is 254 V / (A 2^shift)."""
    a = v.abs().amax(dim=1, keepdim=True)
    V, ev = torch.frexp(v.double())
    A, ea = torch.frexp(a.double())
    V, A = (V * 256).long(), (A * 256).long()
    shift = ea.long() - ev.long()
    den = A << shift.clamp(0, 40)                      # beyond 40 the quotient is far below 1/2 either way
    num = 254 * V.abs() + den
    q = num // (2 * den)
    tie = num % (2 * den) == 0
    return torch.sign(V) * (q - (tie & (q % 2 == 1)).long()), int(tie.sum())


# ------------------------------------------------------------------------------------------- quantiser
@pytest.mark.gpu
@pytest.mark.parametrize("K", [9, 256, 1000, 5001, 7168, 16384, 20001])
@pytest.mark.parametrize("scale", [1.5, 1e-36])
def test_every_integer_of_a_bf16_row_is_the_nearest_half_to_even(K, scale):
    """Elements of half the maximum are 63.5 and go to 64, whatever the maximum."""
    g = rng(30, K)
    v = (normal(g, 128, K).float() * scale).to(torch.bfloat16)
    for r in range(128):                               # rows of every 8-bit maximum, and half of it
        v[r, :4] = torch.tensor([1.0, -0.5, 0.5, 0.25]) * ((128 + r) / 16 * scale)
    v[:, 4:] = v[:, 4:].clamp(-7 * scale, 7 * scale)
    v = v.cuda()
    q, s = rows_out(128, K)
    skg.skg_quantize_q8(v, None, q, s)
    want, ties = nearest_even(v)
    assert ties >= 256
    assert int((q.long() != want).sum()) == 0
