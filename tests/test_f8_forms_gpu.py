"""The quantiser's forms for many blocks: a warp takes 8 or 16 blocks of a row where
there are at least 19456 blocks and rows leave few places over, 16 only of
aligned rows without a gate, 8 of those and of one of the two.  Each form by its
sizes, on either side of those, gated, by an index, and both."""
import pytest
import torch

from projection_gemm_gb300 import build, skg
from tests import f8_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    skg.load()


def normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16).cuda()


def rows_out(M, K):
    return torch.full((M, K), 9.0, device="cuda").to(R.F8), torch.full((M, R.blocks(K)), -1.0, device="cuda")


# blocks a row, groups of 8 blocks: 16 in 2 groups, 23 in 3, 128 in 16; 19456 blocks and one row fewer; 17 leave 7 of 24
# places over, and go by 4
@pytest.mark.parametrize("M,K", [(1216, 2048), (1215, 2048), (846, 2944), (152, 16384), (4096, 16384), (3001, 1024), (1300, 2176)])
def test_gated_rows(M, K):
    g = torch.Generator().manual_seed(M + K)
    both = normal(g, M, 2 * K, std=2.0)
    gate, x = both[:, :K], both[:, K:]
    gate[0, 0], x[0, 0] = -100.0, 2.0 ** 120
    gate[M - 1, K - 1], x[M - 1, K - 2] = 300.0, 0.0
    q, s = rows_out(M, K)
    skg.skg_quantize_f8(x, gate, q, s)
    R.check_gated(x, gate, q, s)


# 16 blocks a warp (7168, 2048 columns), 8 (2944; 7169 of any alignment), 4 (2945 of any alignment: too few rows)
@pytest.mark.parametrize("T,M,K", [(60, 400, 7168), (60, 347, 7168), (100, 1500, 2048), (90, 900, 2944), (60, 400, 7169),
                                   (50, 300, 2945), (4096, 32768, 512)])
@pytest.mark.parametrize("gated", [False, True])
def test_rows_by_an_index(T, M, K, gated):
    g = torch.Generator().manual_seed(T + M + K)
    both = normal(g, T, 2 * K, std=1.5)
    gate, x = (both[:, :K], both[:, K:]) if gated else (None, normal(g, T, K))
    rows = torch.randint(-1, T + 1, (M,), generator=g, dtype=torch.int32)
    rows[0], rows[M - 1], rows[M // 2] = -2 ** 31, 2 ** 31 - 1, T - 1
    q, s = rows_out(M, K)
    skg.skg_quantize_f8(x, gate, q, s, rows=rows.cuda())
    live = ((rows >= 0) & (rows < T)).cuda()
    at = rows.cuda()[live].long()
    if gated:
        R.check_gated(x[at], gate[at], q[live], s[live])
    else:
        R.check_quantised(x[at], q[live], s[live])
    assert bool((q[~live].float() == 0).all()) and bool((s[~live] == 0).all()) and bool((~live).any())


@pytest.mark.parametrize("M,K", [(400, 7168), (348, 7168), (347, 7168), (846, 2944), (400, 7169)])
def test_special_values_in_every_block_of_a_warp(M, K):
    """Not finite, zero, smallest and largest blocks beside each other, in all the places that a warp's blocks have."""
    x = normal(torch.Generator().manual_seed(M), M, K)
    for r in range(1, 12):
        for b in range(r % 5, R.blocks(K), 5):
            e = slice(128 * b, 128 * b + 128)
            v = (0.0, 2.0 ** -133, 3.3895313892515355e38, float("inf"), float("nan"))[(r + b) % 5]
            if (r + b) % 5 < 3:
                x[r, e] = v
            else:
                x[r, min(K - 1, 128 * b + 7 * r)] = v
    q, s = rows_out(M, K)
    skg.skg_quantize_f8(x, None, q, s)
    R.check_quantised(x, q, s)


@pytest.mark.parametrize("M,K,tall", [(512, 7168, 1), (300, 2051, 1), (1001, 1040, 128)])
def test_numbers_are_the_nearest_to_the_exact_quotient_but_for_ties(M, K, tall):
    """Of v 448 / max, in 64 bits.  In steps of e4m3 it is 448 V / (A 2^m), V and A of 8 bits: half way between two
    numbers, or at least 1 / (2 A 2^m) off that, which is above 1e-8 wherever a number that is not 0 is near.  The fp32
    product is off by 2 units of 2^-24, so only a tie T can fall on the other side: where 448 / max is rounded by d and
    the product's exact T (1 + d) is half a unit or more from T.  (That goes by the maximum: of one block no tie may, or
    a good part of them, so there is no share to hold them to.)"""
    v = normal(torch.Generator().manual_seed(M + K), M, K, std=1.5)
    q = torch.empty(M, K, dtype=R.F8, device="cuda")
    mb, kb = -(-M // tall), R.blocks(K)
    s = torch.empty(mb, kb, device="cuda")
    if tall > 1:
        skg.skg_quantize_f8_weights(v, q, s)
    else:
        skg.skg_quantize_f8(v, None, q, s)
    pad = torch.nn.functional.pad(v.double(), (0, kb * 128 - K, 0, mb * tall - M)).view(mb, tall, kb, 128)
    t = (pad * 448 / pad.abs().amax(dim=(1, 3), keepdim=True)).view(mb * tall, kb * 128)[:M, :K]
    steps = t / R.step(t)
    tie = (steps - steps.floor() - 0.5).abs() < 1e-10
    off = (q.double() - t).abs() > R.step(t) * (0.5 + 1e-10)
    assert not bool(off.any())                              # a tie gives either neighbour
    wrong = (q.double() - R.e4m3(t)) != 0
    assert bool((tie | ~wrong).all()) and 0 < int(tie.sum()) < M * K // 50
