"""The tiles that a launch by experts provides for, against the most that offsets can
ask for: with K split a cluster takes one tile, so one too few would leave outputs
unwritten."""
import functools

import pytest
import torch

from projection_gemm_gb300 import build, skg
from tests import f8_reference as R

SMS = 152


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    skg.load()


@functools.lru_cache(maxsize=None)
def most(experts, rows, m_tile):
    """The most token tiles of `rows` rows over `experts` experts, each of whole tiles but its last, by trying every
    number of rows of the last expert."""
    if experts == 1:
        return -(-rows // m_tile)
    return max(most(experts - 1, rows - n, m_tile) + -(-n // m_tile) for n in range(rows + 1))


def ctas_a_tile(d):
    return (2 if d["m_tile"] == 256 else 1) * d["split_k"]


def check_tiles(d, worst):
    n_tiles = -(-d["N"] // d["n_tile"])
    assert d["tiles"] >= worst * n_tiles
    if d["split_k"] > 1:
        assert d["grid"] == ctas_a_tile(d) * d["tiles"]
    else:
        assert 1 <= d["grid"] <= ctas_a_tile(d) * d["tiles"] and d["grid"] % ctas_a_tile(d) == 0


@pytest.mark.parametrize("experts", [1, 2, 5, 9])
def test_planned_tiles_are_enough_for_any_offsets(experts):
    """By trying all of them, at sizes whose launches have every tile of tokens and K split and whole."""
    seen = set()
    for rows in (1, 2, 16, 17, 33, 40, 65, 96, 130, 200):
        for N, K in ((64, 4096), (300, 1024), (2000, 512), (40000, 256), (400000, 1024)):
            d = skg.skg_f8_plan_query(rows, N, K, "bf16", experts, SMS)
            check_tiles(d, most(experts, rows, d["m_tile"]))
            seen.add((d["m_tile"], d["split_k"] > 1))
    assert {m for m, _ in seen} >= {16, 32, 64} and {s for _, s in seen} == {False, True}


@pytest.mark.parametrize("experts", [1, 7, 60, 384, 1024])
@pytest.mark.parametrize("rows", [1, 3, 17, 1000, 5000, 100000, 1 << 20])
def test_planned_tiles_are_enough_for_the_worst_offsets(rows, experts):
    """As many experts as there are with one row each, and whole tiles beyond that."""
    for N, K in ((40, 4096), (300, 1024), (2000, 512)):
        d = skg.skg_f8_plan_query(rows, N, K, "bf16", experts, SMS)
        ones = min(rows, experts)
        check_tiles(d, ones + (rows - ones) // d["m_tile"])


@pytest.mark.gpu
@pytest.mark.parametrize("kind,m_tile,split", [(1, 16, 1), (1, 16, 2), (1, 32, 5), (1, 64, 8), (2, 128, 1), (2, 128, 3),
                                               (2, 256, 1), (2, 256, 4)])
@pytest.mark.parametrize("long", [0, 3, 6])
def test_offsets_that_ask_for_every_tile(kind, m_tile, split, long):
    """One row for each expert but one, which has `long` tiles and a row: as many tiles as there can be, all written."""
    E, N, K = 7, 300, 1024
    counts = [1] * E
    counts[long] += 3 * m_tile
    M = sum(counts)
    plan = skg.F8Plan(M, N, K, "bf16", experts=E)
    plan.force(kind, m_tile, split)
    d = plan.info()
    assert (d["m_tile"], d["split_k"]) == (m_tile, split)
    check_tiles(d, E + 3)
    g = torch.Generator().manual_seed(M)
    x, W = ((torch.randn(*s, generator=g) * 100).clamp(-448, 448).to(R.F8).cuda() for s in ((M, K), (E, N, K)))
    xs, ws = torch.rand(M, 8, generator=g).cuda(), torch.rand(E, 3, 8, generator=g).cuda()
    offsets = torch.tensor([0, *counts]).cumsum(0).int().cuda()
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    plan.run(x, xs, W, ws, None, y, offsets=offsets)
    plan.check()
    at = offsets.tolist()
    for e in range(E):
        s = slice(at[e], at[e + 1])
        R.check_linear(x[s], xs[s], W[e], ws[e], None, y[s])
    plan.close()
