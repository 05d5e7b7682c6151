"""The 8-bit path's host side without a GPU: the plan query's limits and the
refusals of every entry point (each is refused before anything is launched)."""
import ctypes

import pytest

from projection_gemm_gb300 import build, skg

SMS = 152
FAKE = 1 << 20          # an address that is never read: the calls below are refused or launch nothing


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    skg.load()


@pytest.mark.parametrize("args,status", [
    ((0, 128, 128, "bf16", SMS), skg.SKG_ERR_INVALID_ARG),
    ((4, 0, 128, "bf16", SMS), skg.SKG_ERR_INVALID_ARG),
    ((4, 128, 128, 3, SMS), skg.SKG_ERR_INVALID_ARG),
    ((4, 128, 128, -1, SMS), skg.SKG_ERR_INVALID_ARG),
    ((4, 128, 128, "bf16", 0), skg.SKG_ERR_INVALID_ARG),
    ((4, 128, 0, "bf16", SMS), skg.SKG_ERR_UNSUPPORTED),
    ((4, 128, 24, "bf16", SMS), skg.SKG_ERR_UNSUPPORTED),
    ((4, 128, 131072, "bf16", SMS), skg.SKG_ERR_UNSUPPORTED),
    (((1 << 18) + 1, 128, 128, "bf16", SMS), skg.SKG_ERR_UNSUPPORTED),
])
def test_query_refusals(args, status):
    with pytest.raises(skg.SkgError) as e:
        skg.skg_q8_plan_query(*args)
    assert e.value.status == status and skg.skg_last_error()


@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (64, 7168, 7168), (1 << 18, 3, 131056)])
def test_query_limits_are_inside(M, N, K):
    d = skg.skg_q8_plan_query(M, N, K, "fp32", SMS)
    assert (d["M"], d["N"], d["K"], d["epilogue"]) == (M, N, K, skg.SKG_EPI_FP32)


def _norm(M=2, K=8, eps=1e-6, x=FAKE, ldx=8, r=None, ldr=0, gamma=None, h=None, ldh=0, y=None, q=FAKE, s=FAKE):
    return skg.load().skg_rmsnorm_q8(M, K, eps, x, ldx, r, ldr, gamma, h, ldh, y, q, s, None)


def _quant(M=2, K=8, x=FAKE, ldx=8, g=None, ldg=0, q=FAKE, s=FAKE):
    return skg.load().skg_quantize_q8(M, K, x, ldx, g, ldg, q, s, None)


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(K=0), dict(x=None), dict(q=None), dict(s=None), dict(ldx=7), dict(eps=-1.0),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(h=FAKE, ldh=8), dict(r=FAKE, ldr=7),
    dict(r=FAKE, ldr=8, h=FAKE, ldh=7),
])
def test_norm_refuses(kw):
    assert _norm(**kw) == skg.SKG_ERR_INVALID_ARG
    assert "skg_rmsnorm_q8" in skg.skg_last_error()


@pytest.mark.parametrize("kw", [
    dict(x=FAKE + 1), dict(s=FAKE + 2), dict(r=FAKE + 1, ldr=8), dict(gamma=FAKE + 1), dict(y=FAKE + 1),
    dict(r=FAKE, ldr=8, h=FAKE + 1, ldh=8),
])
def test_norm_refuses_misaligned(kw):
    assert _norm(**kw) == skg.SKG_ERR_ALIGNMENT


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), skg.SKG_ERR_INVALID_ARG), (dict(K=0), skg.SKG_ERR_INVALID_ARG),
    (dict(x=None), skg.SKG_ERR_INVALID_ARG), (dict(q=None), skg.SKG_ERR_INVALID_ARG),
    (dict(s=None), skg.SKG_ERR_INVALID_ARG), (dict(ldx=7), skg.SKG_ERR_INVALID_ARG),
    (dict(g=FAKE, ldg=7), skg.SKG_ERR_INVALID_ARG), (dict(g=FAKE + 1, ldg=8), skg.SKG_ERR_ALIGNMENT),
    (dict(x=FAKE + 1), skg.SKG_ERR_ALIGNMENT),
])
def test_quantize_refuses(kw, status):
    assert _quant(**kw) == status


def test_no_rows_launch_nothing():
    assert _norm(M=0) == skg.SKG_OK and _norm(M=0, x=None, q=None, s=None) == skg.SKG_OK
    assert _quant(M=0) == skg.SKG_OK


def test_plan_handles_are_checked():
    lib = skg.load()
    assert lib.skg_q8_run(None, FAKE, FAKE, FAKE, FAKE, None, FAKE, None) == skg.SKG_ERR_INVALID_ARG
    assert lib.skg_q8_plan(4, 128, 128, 0, 0, None) == skg.SKG_ERR_INVALID_ARG
    assert lib.skg_q8_plan_query(4, 128, 128, 0, SMS, None) == skg.SKG_ERR_INVALID_ARG
    assert lib.skg_q8_plan_destroy(None) == skg.SKG_OK
    h = ctypes.c_void_p(FAKE)
    assert lib.skg_q8_plan(4, 128, 20, 0, 0, ctypes.byref(h)) == skg.SKG_ERR_UNSUPPORTED
    assert h.value is None


def test_binding_refuses_host_tensors():
    import torch
    x = torch.zeros(2, 32, dtype=torch.bfloat16)
    q, s = torch.zeros(2, 32, dtype=torch.int8), torch.zeros(2)
    for call in (lambda: skg.skg_rmsnorm_q8(x, None, None, 1e-6, None, q, s),
                 lambda: skg.skg_quantize_q8(x, None, q, s)):
        with pytest.raises(skg.SkgError) as e:
            call()
        assert e.value.status == skg.SKG_ERR_INVALID_ARG


@pytest.mark.parametrize("M,N,K", [(1, 1024, 1024), (3, 384, 7168), (16, 7168, 7168), (64, 7168, 16384), (65, 640, 16),
                                   (40, 40000, 2048), (333, 5001, 4112), (4096, 12288, 7168), (1 << 18, 128, 48)])
def test_query_describes_a_launch_that_covers_every_tile(M, N, K):
    d = skg.skg_q8_plan_query(M, N, K, "bf16", SMS)
    assert d["grid"] >= 1 and d["threads"] % 32 == 0
    assert (d["kernel"] == "q8_stream") == (M <= 8 or M <= 16 and (-(-N // 16) <= 3 * SMS or N * K <= 1 << 24))
    assert d["tiles"] == -(-N // d["n_tile"]) * -(-M // d["m_tile"])
    if d["kernel"] == "q8_stream":
        assert d["workspace_bytes"] == 0 and d["grid"] == d["tiles"] and M <= d["m_tile"]
        return
    nkb = -(-K // 128)
    assert d["smem_bytes"] * d["ctas_per_sm"] <= 227 * 1024
    if d["kernel"] == "q8_split":
        assert d["m_tile"] in ((32,) if M <= 32 else (32, 64)) and 1 <= d["split_k"] <= min(8, nkb) and d["grid"] == d["tiles"] * d["split_k"]
        assert d["split_k"] == 1 or d["grid"] <= SMS * d["ctas_per_sm"]
        put_away = max(0, -(-(-(-nkb // d["split_k"])) // 8) - 2)
        assert d["workspace_bytes"] == d["grid"] * put_away * d["m_tile"] * 512
    else:
        assert 1 <= d["split_k"] <= min(4, nkb)
        assert d["grid"] == 2 * (min(d["tiles"], SMS // 2) if d["split_k"] == 1 else d["split_k"] * d["tiles"])
        assert d["grid"] <= SMS
        assert d["workspace_bytes"] == 0


@pytest.mark.parametrize("M", [1, 8, 9, 16])
@pytest.mark.parametrize("N", [1, 384, 16 * SMS, 16 * SMS + 1, 32 * SMS, 32 * SMS + 1, 48 * SMS, 48 * SMS + 1, 12288, 200000])
def test_streaming_launch_fills_as_few_slots_as_hold_it(M, N):
    d = skg.skg_q8_plan_query(M, N, 7168, "bf16", SMS)
    groups = -(-N // 16)
    if groups <= 3 * SMS:
        assert d["kernel"] == "q8_stream" and d["n_tile"] == 16 and d["ctas_per_sm"] == -(-groups // SMS)
    elif M <= 8:
        assert d["kernel"] == "q8_stream" and d["n_tile"] == 32
    else:
        assert d["kernel"] != "q8_stream"
    assert d["threads"] * d["ctas_per_sm"] <= 1024


@pytest.mark.parametrize("M,N,K,kernel", [
    (16, 7168, 7168, "q8_stream"), (16, 12288, 7168, "q8_split"), (16, 12288, 1024, "q8_stream"), (8, 28672, 8192, "q8_stream"), (17, 7168, 7168, "q8_split"), (64, 7168, 16384, "q8_split"), (64, 28672, 8192, "q8_wide"), (128, 384, 7168, "q8_split"),
    (128, 7168, 7168, "q8_wide"), (256, 4096, 4096, "q8_wide"), (128, 4096, 4096, "q8_split"), (333, 5001, 4112, "q8_wide"), (1000, 4096, 4096, "q8_wide"),
    (65, 7168, 16384, "q8_wide"), (4096, 12288, 7168, "q8_wide")])
def test_batches_take_the_kernel_measured_faster(M, N, K, kernel):
    """Few tiles: K split over clusters; many: whole tiles."""
    assert skg.skg_q8_plan_query(M, N, K, "bf16", SMS)["kernel"] == kernel


@pytest.mark.parametrize("M,N,K,kernel,split", [
    (32, 128 * 36, 7168, "q8_split", 8), (32, 128 * 38, 7168, "q8_split", 7), (32, 128 * 43, 7168, "q8_split", 6),
    (64, 128 * 46, 7168, "q8_split", 6), (64, 128 * 56, 7168, "q8_split", 5), (64, 128 * 59, 2048, "q8_split", 4),
    (128, 256 * 28, 7168, "q8_wide", 2), (128, 256 * 36, 7168, "q8_wide", 2), (128, 256 * 37, 7168, "q8_wide", 1),
    (128, 256 * 23, 16384, "q8_wide", 3), (128, 256 * 24, 16384, "q8_wide", 2), (128, 256 * 32, 2048, "q8_split", 1), (300, 256 * 32, 2048, "q8_wide", 1)])
def test_clusters_of_a_split_k_are_resident_at_once(M, N, K, kernel, split):
    d = skg.skg_q8_plan_query(M, N, K, "bf16", SMS)
    assert (d["kernel"], d["split_k"]) == (kernel, split)
