"""The 8-bit floating point path on a GB300 against its definition in 64 bits
(f8_reference states the bounds): the quantisers over row lengths, strides,
alignments and special values, and the projection over batches, ragged sizes,
launch shapes and distributions of rows over experts."""
import pytest
import torch

from projection_gemm_gb300 import skg
from tests import f8_reference as R

pytestmark = pytest.mark.gpu

LAUNCHES = [(skg.SKG_F8_KERNEL_SPLIT, mt, s) for mt in (16, 32, 64) for s in (1, 2, 5, 8)] + \
           [(skg.SKG_F8_KERNEL_WIDE, mt, s) for mt in (128, 256) for s in (1, 2, 3, 4)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from projection_gemm_gb300 import build
    build.build()
    skg.load()
    assert torch.cuda.is_available()


def gen(*key):
    seed = 0
    for k in key:
        seed = seed * 1000003 + int(k)
    return torch.Generator().manual_seed(seed % 2 ** 31)


def normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16).cuda()


def numbers(g, *shape):
    return (torch.randn(*shape, generator=g) * 160).clamp(-448, 448).to(R.F8).cuda()


def positive(g, *shape, mean=1.0):
    return (mean * (0.5 + torch.rand(*shape, generator=g))).cuda()


def rows_out(M, K):
    q = torch.full((M, K), 9.0, device="cuda").to(R.F8)
    return q, torch.full((M, R.blocks(K)), -1.0, device="cuda")


# ------------------------------------------------------------------------------------------------ quantiser
@pytest.mark.parametrize("M", [1, 5, 300, 3001])
@pytest.mark.parametrize("K", [1, 7, 8, 127, 128, 129, 136, 144, 256, 300, 384, 400, 1000, 1024, 1032, 1040, 2048, 4112, 5001,
                               7168])
def test_quantise_rows(M, K):
    g = gen(1, M, K)
    x = normal(g, M, K, std=1.5)
    q, s = rows_out(M, K)
    skg.skg_quantize_f8(x, None, q, s)
    R.check_quantised(x, q, s)


@pytest.mark.parametrize("K,ld,off", [(1000, 1000, 1), (1000, 1024, 0), (1024, 1031, 3), (4096, 8192, 4096), (333, 335, 5)])
def test_quantise_strides_and_offsets(K, ld, off):
    g = gen(2, K, ld)
    M = 9
    big = normal(g, M * ld + off + K)
    x = big[off:off + M * ld].as_strided((M, K), (ld, 1))
    q, s = rows_out(M, K)
    skg.skg_quantize_f8(x, None, q, s)
    R.check_quantised(x.contiguous(), q, s)


@pytest.mark.parametrize("M,K", [(3, 5), (17, 640), (64, 1003), (300, 4096), (1000, 208), (2001, 2064), (1500, 2051), (9, 48)])
def test_quantise_gated_halves_of_one_tensor(M, K):
    g = gen(3, M, K)
    both = normal(g, M, 2 * K, std=2.0)
    gate, x = both[:, :K], both[:, K:]
    gate[0, 0] = -100.0                       # exp leaves fp32's normal range; the product need not
    x[0, 0] = 2.0 ** 120
    q, s = rows_out(M, K)
    skg.skg_quantize_f8(x, gate, q, s)
    R.check_gated(x, gate, q, s)


@pytest.mark.parametrize("T,K", [(5, 128), (40, 1000), (64, 4097)])
@pytest.mark.parametrize("gated", [False, True])
def test_quantise_by_rows(T, K, gated):
    """Rows taken by an index: any order, one more than once, and none where the index is of no row."""
    g = gen(4, T, K)
    x, gate = normal(g, T, K), normal(g, T, K) if gated else None
    rows = torch.randint(-2, T + 2, (3 * T + 1,), generator=g, dtype=torch.int32)
    rows[0], rows[1], rows[2] = -2 ** 31, 2 ** 31 - 1, T
    q, s = rows_out(len(rows), K)
    skg.skg_quantize_f8(x, gate, q, s, rows=rows.cuda())
    q0, s0 = rows_out(T, K)
    skg.skg_quantize_f8(x, gate, q0, s0)
    live = (rows >= 0) & (rows < T)
    at = rows[live].long().cuda()
    live = live.cuda()
    assert torch.equal(q[live].float(), q0[at].float()) and torch.equal(s[live], s0[at])
    assert bool((q[~live].float() == 0).all()) and bool((s[~live] == 0).all())


@pytest.mark.parametrize("K", [128, 131, 1024])
def test_quantise_special_values(K):
    x = normal(gen(5, K), 12, K)
    x[0] = 0
    x[1, 3] = float("inf")
    x[2, 5] = float("nan")
    x[3, 0] = float("-inf")
    x[4] = 2.0 ** -133                        # bf16's smallest
    x[5] = 3.3895313892515355e38              # its largest
    x[6] = 2.0 ** -126
    x[7] *= 2.0 ** -120
    x[8] = -0.0
    x[9, :] = 1.0
    x[10, 1:] *= 2.0 ** -30                   # all but one of the first block below e4m3's smallest
    q, s = rows_out(12, K)
    skg.skg_quantize_f8(x, None, q, s)
    R.check_quantised(x, q, s)
    assert bool(s[1, 0].isnan()) and bool((q[1, :128].float() == 0).all())


@pytest.mark.parametrize("E,N,K", [(1, 1, 1), (1, 128, 128), (1, 129, 136), (1, 300, 1003), (3, 200, 256), (2, 5, 4112)])
def test_quantise_weights(E, N, K):
    W = normal(gen(6, E, N, K), E, N, K, std=0.02)
    W[0, -1, -1] = float("nan") if N == 129 else 3.0
    q = torch.full(W.shape, 9.0, device="cuda").to(R.F8)
    s = torch.full((E, R.blocks(N), R.blocks(K)), -1.0, device="cuda")
    if E == 1:
        skg.skg_quantize_f8_weights(W[0], q[0], s[0])
    else:
        skg.skg_quantize_f8_weights(W, q, s)
    for e in range(E):
        R.check_quantised(W[e], q[e], s[e], R.BLOCK)


# ----------------------------------------------------------------------------------------------- projection
def operands(g, M, N, K, E=0):
    each = (E,) if E else ()
    return (numbers(g, M, K), positive(g, M, R.blocks(K), mean=1 / 160), numbers(g, *each, N, K),
            positive(g, *each, R.blocks(N), R.blocks(K), mean=1 / 160))


def project(M, N, K, epilogue, launch=None, static=False, seed=0):
    g = gen(7, M, N, K, seed)
    x, xs, W, ws = operands(g, M, N, K)
    res = normal(g, M, N) if epilogue == "bf16_residual" else None
    y = torch.full((M, N), float("nan"), device="cuda", dtype=torch.float32 if epilogue == "fp32" else torch.bfloat16)
    plan = skg.F8Plan(M, N, K, epilogue, static_weights=static)
    if launch:
        plan.force(*launch)
    plan.run(x, xs, W, ws, res, y)
    plan.check()
    R.check_linear(x, xs, W, ws, res, y, f"{M}x{N}x{K} {epilogue} {launch or plan.info()}")
    plan.close()


@pytest.mark.parametrize("launch", LAUNCHES)
@pytest.mark.parametrize("M,N,K,epilogue", [(1, 128, 128, "fp32"), (16, 300, 1024, "bf16"), (130, 257, 1552, "bf16_residual"),
                                            (300, 130, 400, "fp32")])
def test_projection_by_every_launch(launch, M, N, K, epilogue):
    project(M, N, K, epilogue, launch)


@pytest.mark.parametrize("epilogue", ["bf16", "bf16_residual", "fp32"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 7168, 7168), (2, 5, 48), (7, 384, 7168), (17, 1000, 144), (64, 640, 16384),
                                   (65, 333, 2064), (256, 512, 512), (257, 129, 272), (1000, 2048, 1024), (2049, 776, 4112)])
def test_projection_as_planned(M, N, K, epilogue):
    project(M, N, K, epilogue, static=M % 2 == 1)


def by_experts(counts, N, K, epilogue="bf16", launch=None, first=0, behind=0, seed=0):
    """Rows first .. of the experts in turn; those before and behind them are nobody's and stay as they were."""
    E, M = len(counts), first + sum(counts) + behind
    g = gen(8, M, N, K, seed)
    x, xs, W, ws = operands(g, M, N, K, E)
    res = normal(g, M, N) if epilogue == "bf16_residual" else None
    offsets = torch.tensor([first, *counts]).cumsum(0).to(torch.int32).cuda()
    out = torch.float32 if epilogue == "fp32" else torch.bfloat16
    y = torch.full((M, N), -7.0, device="cuda", dtype=out)
    plan = skg.F8Plan(M, N, K, epilogue, experts=E)
    if launch:
        plan.force(*launch)
    plan.run(x, xs, W, ws, res, y, offsets=offsets)
    plan.check()
    at = offsets.tolist()
    for e in range(E):
        a, b = at[e], at[e + 1]
        if b > a:
            R.check_linear(x[a:b], xs[a:b], W[e], ws[e], None if res is None else res[a:b], y[a:b],
                           f"expert {e} of {counts} {launch or plan.info()}")
    assert bool((y[:first] == -7).all()) and bool((y[at[-1]:] == -7).all())
    plan.close()


@pytest.mark.parametrize("launch", LAUNCHES)
@pytest.mark.parametrize("counts,N,K", [([3], 130, 256), ([0, 1, 0, 17, 130, 0], 200, 400), ([300, 0, 5, 256], 129, 1040)])
def test_experts_by_every_launch(launch, counts, N, K):
    by_experts(counts, N, K, launch=launch, behind=3)


@pytest.mark.parametrize("epilogue", ["bf16", "bf16_residual", "fp32"])
@pytest.mark.parametrize("counts,first,behind", [([1], 0, 0), ([0, 0, 0, 2], 0, 0), ([0] * 40, 0, 5), ([2, 0, 1] * 100, 0, 9),
                                                 ([1] * 1024, 0, 0), ([700, 1, 0, 300], 11, 0), ([64] * 20, 0, 100)])
def test_experts_as_planned(counts, first, behind, epilogue):
    by_experts(counts, 136, 272, epilogue, first=first, behind=behind)


@pytest.mark.parametrize("launch", [(1, 16, 1), (1, 32, 2), (2, 128, 1), (2, 256, 1)])
@pytest.mark.parametrize("offsets", [[-5, 3, 2, 900, 20], [30, 20, 10, 0, -1], [0, 0, 0, 0, 2 ** 31 - 1],
                                     [-2 ** 31, -1, 5, 4, 40]])
def test_offsets_that_are_out_of_order_or_range(offsets, launch):
    """They are held to [0, M] and to ascend: no access leaves its tensor, and the rows of those ranges are projected."""
    g = gen(9)
    M, N, K = 40, 130, 256
    x, xs, W, ws = operands(g, M, N, K, 4)
    y = torch.full((M, N), -7.0, device="cuda", dtype=torch.bfloat16)
    plan = skg.F8Plan(M, N, K, "bf16", experts=4)
    plan.force(*launch)
    plan.run(x, xs, W, ws, None, y, offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    plan.check()
    at, top = [], 0
    for o in offsets:
        top = max(top, min(max(o, 0), M))
        at.append(top)
    for e in range(4):
        a, b = at[e], at[e + 1]
        if b > a:
            R.check_linear(x[a:b], xs[a:b], W[e], ws[e], None, y[a:b])
    assert bool((y[:at[0]] == -7).all()) and bool((y[at[4]:] == -7).all())


@pytest.mark.parametrize("launch", [(1, 16, 4), (1, 64, 1), (2, 128, 3), (2, 256, 1)])
def test_scales_that_are_nan_or_zero_stay_in_their_rows_and_blocks(launch):
    g = gen(10)
    M, N, K = 40, 300, 512
    x, xs, W, ws = operands(g, M, N, K)
    xs[3, 1] = float("nan")
    xs[4] = 0
    ws[1, 2] = float("nan")
    y = torch.empty(M, N, device="cuda")
    plan = skg.F8Plan(M, N, K, "fp32")
    plan.force(*launch)
    plan.run(x, xs, W, ws, None, y)
    plan.check()
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[3] = True
    bad[:, 128:256] = True
    assert bool((y.isnan() == bad).all())
    assert bool((y[4, :128] == 0).all())
    ok = torch.ones(M, dtype=torch.bool, device="cuda")
    ok[3] = False
    R.check_linear(x[ok], xs[ok], W[:128], ws[:1], None, y[ok][:, :128])
