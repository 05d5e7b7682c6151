"""The 8-bit floating point path's and the experts' host side without a GPU: the
plan query's limits and choices, and the refusals of every entry point (each is
refused before anything is launched)."""
import ctypes

import pytest

from projection_gemm_gb300 import build, skg

SMS = 152
FAKE = 1 << 20          # an address that is never read: the calls below are refused or launch nothing
BIG = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    skg.load()


@pytest.mark.parametrize("args,status", [
    ((0, 128, 128, "bf16", 0, SMS), skg.SKG_ERR_INVALID_ARG),
    ((4, 0, 128, "bf16", 0, SMS), skg.SKG_ERR_INVALID_ARG),
    ((4, 128, 128, 3, 0, SMS), skg.SKG_ERR_INVALID_ARG),
    ((4, 128, 128, -1, 0, SMS), skg.SKG_ERR_INVALID_ARG),
    ((4, 128, 128, "bf16", -1, SMS), skg.SKG_ERR_INVALID_ARG),
    ((4, 128, 128, "bf16", 0, 0), skg.SKG_ERR_INVALID_ARG),
    ((4, 128, 0, "bf16", 0, SMS), skg.SKG_ERR_UNSUPPORTED),
    ((4, 128, 24, "bf16", 0, SMS), skg.SKG_ERR_UNSUPPORTED),
    ((4, 128, 131088, "bf16", 0, SMS), skg.SKG_ERR_UNSUPPORTED),
    (((1 << 20) + 1, 128, 128, "bf16", 0, SMS), skg.SKG_ERR_UNSUPPORTED),
    ((4, 128, 128, "bf16", 1025, SMS), skg.SKG_ERR_UNSUPPORTED),
    ((4, BIG, 128, "bf16", 0, SMS), skg.SKG_ERR_UNSUPPORTED),
    ((4, 1 << 22, 128, "bf16", 1024, SMS), skg.SKG_ERR_UNSUPPORTED),
    ((1 << 20, 1 << 30, 128, "bf16", 0, SMS), skg.SKG_ERR_UNSUPPORTED),
    ((2 ** 32 + 16, 128, 128, "bf16", 0, SMS), skg.SKG_ERR_INVALID_ARG),
])
def test_query_refusals(args, status):
    with pytest.raises(skg.SkgError) as e:
        skg.skg_f8_plan_query(*args)
    assert e.value.status == status and str(e.value)


@pytest.mark.parametrize("M,N,K,E", [(1, 1, 16, 0), (64, 7168, 7168, 0), (1 << 20, 3, 131072, 0), (1, 1, 16, 1024),
                                     (1 << 20, 128, 128, 1024), (8, 2 ** 31 - 256, 16, 0)])
def test_query_limits_are_inside(M, N, K, E):
    d = skg.skg_f8_plan_query(M, N, K, "fp32", E, SMS)
    assert (d["M"], d["N"], d["K"], d["epilogue"], d["experts"]) == (M, N, K, skg.SKG_EPI_FP32, E)
    assert d["smem_bytes"] * d["ctas_per_sm"] <= 227 * 1024 and d["grid"] >= 1
    pair = 2 if d["m_tile"] == 256 else 1
    assert d["grid"] % (pair * d["split_k"]) == 0
    assert d["grid"] <= (pair * d["split_k"] * d["tiles"] if d["split_k"] > 1 else SMS * d["ctas_per_sm"])


@pytest.mark.parametrize("T", [1, 3, 17, 100, 1000, 5000])
@pytest.mark.parametrize("E", [1, 2, 60, 384, 1024])
@pytest.mark.parametrize("m_tile", [16, 32, 64, 128, 256])
def test_tiles_are_the_most_that_offsets_can_ask_for(T, E, m_tile):
    """Of T rows over E experts: as many experts as can begin a tile with one row, the rest whole tiles."""
    worst = 0
    for ones in range(min(E, T) + 1):                   # experts with one row; the others share the rest
        rest = T - ones
        worst = max(worst, ones + (-(-rest // m_tile) if E > ones else 0))
        if E > ones:                                     # a second one ragged
            worst = max(worst, ones + rest // m_tile + (1 if rest % m_tile else 0))
    assert worst <= min(E, T) + T // m_tile


@pytest.mark.parametrize("M,N,K,E,kind", [(1, 12288, 7168, 0, 1), (64, 7168, 16384, 0, 1), (4096, 12288, 7168, 0, 2),
                                          (128, 2048, 4096, 384, 1), (16384, 4096, 4096, 32, 2)])
def test_kernel_follows_rows(M, N, K, E, kind):
    assert skg.skg_f8_plan_query(M, N, K, "bf16", E, SMS)["kernel_kind"] == kind


def _quant(M=2, K=8, x=FAKE, ldx=8, g=None, ldg=0, rows=None, x_rows=0, q=FAKE, s=FAKE):
    return skg.load().skg_quantize_f8(M, K, x, ldx, g, ldg, rows, x_rows, q, s, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), skg.SKG_ERR_INVALID_ARG), (dict(K=0), skg.SKG_ERR_INVALID_ARG), (dict(x=None), skg.SKG_ERR_INVALID_ARG),
    (dict(q=None), skg.SKG_ERR_INVALID_ARG), (dict(s=None), skg.SKG_ERR_INVALID_ARG),
    (dict(ldx=7), skg.SKG_ERR_INVALID_ARG), (dict(g=FAKE, ldg=7), skg.SKG_ERR_INVALID_ARG),
    (dict(rows=FAKE, x_rows=-1), skg.SKG_ERR_INVALID_ARG), (dict(rows=FAKE, x_rows=1, x=None), skg.SKG_ERR_INVALID_ARG),
    (dict(K=(1 << 30) + 1, ldx=1 << 31), skg.SKG_ERR_UNSUPPORTED),
    (dict(x=FAKE + 1), skg.SKG_ERR_ALIGNMENT), (dict(g=FAKE + 1, ldg=8), skg.SKG_ERR_ALIGNMENT),
    (dict(s=FAKE + 2), skg.SKG_ERR_ALIGNMENT), (dict(rows=FAKE + 2, x_rows=1), skg.SKG_ERR_ALIGNMENT),
    (dict(M=0), skg.SKG_OK), (dict(M=0, x=None, q=None, s=None), skg.SKG_OK),
])
def test_quantise_refuses(kw, status):
    assert _quant(**kw) == status
    assert status == skg.SKG_OK or "skg_quantize_f8" in skg.skg_last_error()


@pytest.mark.parametrize("args,status", [
    ((0, 4, 8, FAKE, FAKE, FAKE), skg.SKG_ERR_INVALID_ARG), ((1, 0, 8, FAKE, FAKE, FAKE), skg.SKG_ERR_INVALID_ARG),
    ((1, 4, 0, FAKE, FAKE, FAKE), skg.SKG_ERR_INVALID_ARG), ((1, 4, 8, None, FAKE, FAKE), skg.SKG_ERR_INVALID_ARG),
    ((1, 4, 8, FAKE, None, FAKE), skg.SKG_ERR_INVALID_ARG), ((1, 4, 8, FAKE, FAKE, None), skg.SKG_ERR_INVALID_ARG),
    ((1, 4, 8, FAKE + 1, FAKE, FAKE), skg.SKG_ERR_ALIGNMENT), ((1, 4, 8, FAKE, FAKE, FAKE + 2), skg.SKG_ERR_ALIGNMENT),
    ((1024, 1 << 20, 1 << 17, FAKE, FAKE, FAKE), skg.SKG_ERR_UNSUPPORTED),
    ((1, 4, (1 << 30) + 8, FAKE, FAKE, FAKE), skg.SKG_ERR_UNSUPPORTED),
])
def test_quantise_weights_refuses(args, status):
    assert skg.load().skg_quantize_f8_weights(*args, None) == status


def test_plan_and_run_refuse_null():
    lib = skg.load()
    assert lib.skg_f8_plan(4, 128, 128, 0, 0, 0, None) == skg.SKG_ERR_INVALID_ARG
    assert lib.skg_f8_plan_query(4, 128, 128, 0, 0, SMS, None) == skg.SKG_ERR_INVALID_ARG
    assert lib.skg_f8_run(None, *[FAKE] * 4, None, None, FAKE, None) == skg.SKG_ERR_INVALID_ARG
    assert lib.skg_f8_plan_force(None, 0, 0, 0) == skg.SKG_ERR_INVALID_ARG
    assert lib.skg_f8_plan_info(None, None) == skg.SKG_ERR_INVALID_ARG
    assert lib.skg_f8_plan_check(None) == skg.SKG_ERR_INVALID_ARG
    assert lib.skg_f8_debug_wait_timeout(None, 1000, None) == skg.SKG_ERR_INVALID_ARG
    assert lib.skg_f8_plan_destroy(None) == skg.SKG_OK
    h = ctypes.c_void_p(1)
    assert lib.skg_f8_plan(0, 128, 128, 0, 0, 0, ctypes.byref(h)) == skg.SKG_ERR_INVALID_ARG and h.value is None


def _sort(T=2, k=2, E=4, e=FAKE, o=FAKE, r=FAKE, p=FAKE):
    return skg.load().skg_experts_sort(T, k, E, e, o, r, p, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), skg.SKG_ERR_INVALID_ARG), (dict(k=0), skg.SKG_ERR_INVALID_ARG), (dict(E=0), skg.SKG_ERR_INVALID_ARG),
    (dict(E=1025), skg.SKG_ERR_UNSUPPORTED), (dict(T=1 << 22, k=5), skg.SKG_ERR_UNSUPPORTED),
    (dict(T=BIG, k=BIG), skg.SKG_ERR_UNSUPPORTED),
    (dict(e=None), skg.SKG_ERR_INVALID_ARG), (dict(o=None), skg.SKG_ERR_INVALID_ARG), (dict(r=None), skg.SKG_ERR_INVALID_ARG),
    (dict(p=None), skg.SKG_ERR_INVALID_ARG), (dict(e=FAKE + 1), skg.SKG_ERR_ALIGNMENT), (dict(p=FAKE + 2), skg.SKG_ERR_ALIGNMENT),
])
def test_sort_refuses(kw, status):
    assert _sort(**kw) == status


def _gather(R=2, T=2, N=8, x=FAKE, ldx=8, rows=FAKE, out=FAKE):
    return skg.load().skg_experts_gather(R, T, N, x, ldx, rows, out, None)


@pytest.mark.parametrize("kw,status", [
    (dict(R=-1), skg.SKG_ERR_INVALID_ARG), (dict(T=-1), skg.SKG_ERR_INVALID_ARG), (dict(N=0), skg.SKG_ERR_INVALID_ARG),
    (dict(x=None), skg.SKG_ERR_INVALID_ARG), (dict(rows=None), skg.SKG_ERR_INVALID_ARG), (dict(out=None), skg.SKG_ERR_INVALID_ARG),
    (dict(ldx=7), skg.SKG_ERR_INVALID_ARG), (dict(N=(1 << 30) + 1, ldx=1 << 31), skg.SKG_ERR_UNSUPPORTED),
    (dict(x=FAKE + 1), skg.SKG_ERR_ALIGNMENT), (dict(rows=FAKE + 2), skg.SKG_ERR_ALIGNMENT), (dict(out=FAKE + 1), skg.SKG_ERR_ALIGNMENT),
    (dict(R=0), skg.SKG_OK),
])
def test_gather_refuses(kw, status):
    assert _gather(**kw) == status


def _combine(T=2, k=2, R=4, N=8, y=FAKE, ldy=8, pos=FAKE, w=FAKE, res=None, out=FAKE):
    return skg.load().skg_experts_combine(T, k, R, N, y, ldy, pos, w, res, out, None)


def _grad(T=2, k=2, R=4, N=8, go=FAKE, y=FAKE, ldy=8, pos=FAKE, w=FAKE, gy=FAKE, gw=FAKE):
    return skg.load().skg_experts_combine_grad(T, k, R, N, go, y, ldy, pos, w, gy, gw, None)


COMMON = [
    (dict(T=-1), skg.SKG_ERR_INVALID_ARG), (dict(k=0), skg.SKG_ERR_INVALID_ARG), (dict(R=-1), skg.SKG_ERR_INVALID_ARG),
    (dict(N=0), skg.SKG_ERR_INVALID_ARG), (dict(T=BIG, k=2), skg.SKG_ERR_UNSUPPORTED),
    (dict(N=(1 << 30) + 1, ldy=1 << 31), skg.SKG_ERR_UNSUPPORTED), (dict(y=None), skg.SKG_ERR_INVALID_ARG),
    (dict(pos=None), skg.SKG_ERR_INVALID_ARG), (dict(ldy=7), skg.SKG_ERR_INVALID_ARG), (dict(y=FAKE + 1), skg.SKG_ERR_ALIGNMENT),
    (dict(pos=FAKE + 2), skg.SKG_ERR_ALIGNMENT), (dict(w=FAKE + 2), skg.SKG_ERR_ALIGNMENT), (dict(T=0), skg.SKG_OK),
]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(out=None), skg.SKG_ERR_INVALID_ARG), (dict(out=FAKE + 1), skg.SKG_ERR_ALIGNMENT), (dict(res=FAKE + 1), skg.SKG_ERR_ALIGNMENT)])
def test_combine_refuses(kw, status):
    assert _combine(**kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(go=None), skg.SKG_ERR_INVALID_ARG), (dict(w=None), skg.SKG_ERR_INVALID_ARG), (dict(gy=None), skg.SKG_ERR_INVALID_ARG),
    (dict(gw=None), skg.SKG_ERR_INVALID_ARG), (dict(gy=FAKE + 1), skg.SKG_ERR_ALIGNMENT), (dict(gw=FAKE + 2), skg.SKG_ERR_ALIGNMENT)])
def test_combine_grad_refuses(kw, status):
    assert _grad(**kw) == status


def test_binding_refuses_tensors_that_do_not_fit():
    """CPU tensors, wrong types and shapes: refused by the binding, before the library is called."""
    import torch
    bf, i32 = torch.bfloat16, torch.int32
    x, rows, out = torch.zeros(4, 8, dtype=bf), torch.zeros(8, dtype=i32), torch.zeros(8, 8, dtype=bf)
    q, s = torch.zeros(4, 8).to(torch.float8_e4m3fn), torch.zeros(4, 1)
    pos, w = torch.zeros(4, 2, dtype=i32), torch.zeros(4, 2)
    calls = [
        lambda: skg.skg_quantize_f8(x, None, q, s),
        lambda: skg.skg_quantize_f8(x[0], None, q, s),
        lambda: skg.skg_quantize_f8_weights(x, q, s),
        lambda: skg.skg_quantize_f8_weights(x[0], q[0], s),
        lambda: skg.skg_experts_sort(pos, torch.zeros(5, dtype=i32), rows, pos),
        lambda: skg.skg_experts_sort(pos[0], torch.zeros(5, dtype=i32), rows, pos),
        lambda: skg.skg_experts_gather(x, rows, out),
        lambda: skg.skg_experts_gather(x, pos, out),
        lambda: skg.skg_experts_combine(out, pos, w, None, x),
        lambda: skg.skg_experts_combine(out, rows, w, None, x),
        lambda: skg.skg_experts_combine_grad(x, out, pos, w, out, w),
    ]
    for call in calls:
        with pytest.raises(skg.SkgError) as e:
            call()
        assert e.value.status == skg.SKG_ERR_INVALID_ARG
