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
