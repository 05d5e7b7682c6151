"""The 8-bit path on a GB300 against its definition in 64 bits (q8_reference
states the bounds): the norm and the quantiser over row lengths, strides,
alignments and special values, and the projection over batches, ragged sizes
and the largest sums, plus streams, graphs and refusals."""
import numpy as np
import pytest
import torch

from projection_gemm_gb300 import skg
from tests import q8_reference as R

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from projection_gemm_gb300 import build
    build.build()
    skg.load()
    assert torch.cuda.is_available()


def rng(*key):
    return np.random.Generator(np.random.PCG64(list(key)))


def normal(g, *shape, std=1.0):
    return torch.from_numpy(g.standard_normal(shape, dtype=np.float32) * np.float32(std)).to(torch.bfloat16)


def rows_out(M, K):
    q = torch.full((M, K), 99, dtype=torch.int8, device="cuda")
    return q, torch.full((M,), float("nan"), dtype=torch.float32, device="cuda")


# ------------------------------------------------------------------------------------------------- norm
@pytest.mark.parametrize("M", [1, 3, 64])
@pytest.mark.parametrize("K", [1, 2, 7, 8, 31, 255, 256, 257, 1000, 1024, 2048, 4099, 5001, 7168, 8192, 8200, 16384,
                               16392, 20001, 40000])
def test_norm_against_64_bits(M, K):
    g = rng(1, M, K)
    x, r, gamma = normal(g, M, K).cuda(), normal(g, M, K, std=2.0).cuda(), (normal(g, K, std=0.25) + 1).cuda()
    q, s = rows_out(M, K)
    h, y = torch.empty_like(x), torch.empty_like(x)
    skg.skg_rmsnorm_q8(x, r, gamma, EPS, h, q, s, y)
    v, _ = R.norm_rows(x, r, gamma, EPS)
    e = R.row_error(K)
    R.check_rows(v, q, s, e, f"norm {M}x{K}")
    assert torch.equal(h, (x.float() + r.float()).to(torch.bfloat16))
    assert bool(((y.double() - v).abs() <= (2.0 ** -8 + e) * v.abs() + 2.0 ** -133).all())


@pytest.mark.parametrize("residual,gamma,h", [(False, True, False), (True, False, True), (True, True, False),
                                              (False, False, False)])
@pytest.mark.parametrize("K", [37, 1024, 7168])
def test_norm_optional_tensors(residual, gamma, h, K):
    g = rng(2, K)
    M = 5
    x = normal(g, M, K).cuda()
    r = normal(g, M, K).cuda() if residual else None
    w = normal(g, K).cuda() if gamma else None
    hh = torch.empty_like(x) if h else None
    q, s = rows_out(M, K)
    skg.skg_rmsnorm_q8(x, r, w, 1e-5, hh, q, s)
    v, _ = R.norm_rows(x, r, w, 1e-5)
    R.check_rows(v, q, s, R.row_error(K))
    if h:
        assert torch.equal(hh, (x.float() + r.float()).to(torch.bfloat16))


@pytest.mark.parametrize("K,ld,off", [(1000, 1000, 1), (1000, 1024, 0), (1024, 1031, 3), (4096, 8192, 4096),
                                      (7168, 7176, 8), (333, 335, 5)])
def test_norm_strides_and_offsets(K, ld, off):
    """Rows inside wider tensors, starting at any element; h in place of the residual."""
    g = rng(3, K, ld)
    M = 9
    big = normal(g, M * ld + off + K).cuda()
    x = big[off:off + M * ld].as_strided((M, K), (ld, 1))
    rbig = normal(g, M, ld + 2).cuda()
    r = rbig[:, 1:1 + K] if ld + 2 > K + 1 else rbig[:, :K]
    before = rbig.clone()
    want_h = (x.float() + r.float()).to(torch.bfloat16)
    v, _ = R.norm_rows(x, r, None, EPS)
    q, s = rows_out(M, K)
    skg.skg_rmsnorm_q8(x, r, None, EPS, r, q, s)
    R.check_rows(v, q, s, R.row_error(K))
    assert torch.equal(r, want_h)
    r.copy_(before[:, 1:1 + K] if ld + 2 > K + 1 else before[:, :K])
    assert torch.equal(rbig, before)                 # nothing beside the rows was written


@pytest.mark.parametrize("K", [5, 256, 7168, 20001])
def test_rows_of_zeros_and_values_that_are_not_finite(K):
    g = rng(4, K)
    x = normal(g, 8, K)
    x[1] = 0
    x[2, K // 2] = float("nan")
    x[3, K - 1] = float("inf")
    x[4, 0] = float("-inf")
    x = x.cuda()
    for call in (lambda q, s: skg.skg_rmsnorm_q8(x, None, None, EPS, None, q, s),
                 lambda q, s: skg.skg_quantize_q8(x, None, q, s)):
        q, s = rows_out(8, K)
        call(q, s)
        assert bool(s[2:5].isnan().all()) and bool((q[2:5] == 0).all())
        assert s[1] == 0 and bool((q[1] == 0).all())
        ok = [0, 5, 6, 7]
        assert bool(s[ok].isfinite().all()) and bool((q[ok].abs().amax(dim=1) == 127).all())


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-20, 1e10, 3e38])
def test_quantize_over_the_exponent_range(scale):
    g = rng(5)
    x = torch.from_numpy(g.uniform(-1, 1, size=(4, 513)) * scale).to(torch.bfloat16).cuda()
    q, s = rows_out(4, 513)
    skg.skg_quantize_q8(x, None, q, s)
    R.check_rows(x.double(), q, s, R.row_error(513), f"values of {scale}")


@pytest.mark.parametrize("scale", [1e-30, 1e15, 1e25, 1e38])
def test_norm_over_the_exponent_range(scale):
    """Squares that leave fp32's range: the norm of finite values stays what it is."""
    g = rng(6)
    x = torch.from_numpy(g.uniform(-1, 1, size=(4, 1000)) * scale).to(torch.bfloat16).cuda()
    q, s = rows_out(4, 1000)
    skg.skg_rmsnorm_q8(x, None, None, EPS, None, q, s)
    v, _ = R.norm_rows(x, None, None, EPS)
    R.check_rows(v, q, s, R.row_error(1000), f"values of {scale}")


# -------------------------------------------------------------------------------------------- quantiser
@pytest.mark.parametrize("M", [1, 6])
@pytest.mark.parametrize("K", [1, 2, 9, 64, 511, 512, 1000, 4096, 5001, 8192, 16384, 16385, 32768, 50000])
@pytest.mark.parametrize("gated", [False, True])
def test_quantize_against_64_bits(M, K, gated):
    g = rng(7, M, K, gated)
    both = normal(g, M, 2 * K, std=1.5).cuda()
    x, gate = both[:, K:], both[:, :K] if gated else None
    q, s = rows_out(M, K)
    skg.skg_quantize_q8(x, gate, q, s)
    R.check_rows(R.gated_rows(x, gate), q, s, R.row_error(K, gate), f"quantize {M}x{K} gated={gated}")


def test_quantize_large_gates():
    """silu far out on both sides: 0 for large negative gates, the gate itself for large positive ones."""
    gate = torch.tensor([[-1e4, -200.0, -89.0, -20.0, 0.0, 20.0, 89.0, 1e4]], dtype=torch.bfloat16, device="cuda")
    x = torch.full_like(gate, 1.0)
    for lo, hi in ((0, 8), (0, 3), (2, 5)):
        gg, xx = gate[:, lo:hi].contiguous(), x[:, lo:hi].contiguous()
        q, s = rows_out(1, hi - lo)
        skg.skg_quantize_q8(xx, gg, q, s)
        v = R.gated_rows(xx, gg)
        if float(v.abs().max()) > 2.0 ** -126:
            R.check_rows(v, q, s, R.row_error(hi - lo, gg))
        else:
            assert bool(s.isfinite().all())


def test_quantize_half_way_values_go_to_the_even_integer():
    x = torch.zeros(1, 256, dtype=torch.bfloat16)
    x[0, 0] = 127
    x[0, 1:8] = torch.tensor([0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 3.5])
    q, s = rows_out(1, 256)
    skg.skg_quantize_q8(x.cuda(), None, q, s)
    assert s.item() == 1.0 and q[0, :8].tolist() == [127, 0, 2, 2, 0, -2, -2, 4]


@pytest.mark.parametrize("gated", [False, True])
def test_rows_beyond_32_bit_offsets(gated):
    """More than 2^32 elements: the last rows are right, each row from its own values."""
    M, K = 270_000, 16_384
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    g = rng(8)
    at = [0, 131_071, 131_072, 262_143, 262_144, M - 1]
    x[at] = normal(g, len(at), K).cuda()
    gate = x if gated else None
    q, s = rows_out(M, K)
    skg.skg_quantize_q8(x, gate, q, s)
    R.check_rows(R.gated_rows(x[at], x[at] if gated else None), q[at], s[at], R.row_error(K, x[at]))
    assert int((s != 0).sum()) == len(at)
    del q
    if not gated:
        q = torch.empty(M, K, dtype=torch.int8, device="cuda")
        skg.skg_rmsnorm_q8(x, x, None, EPS, x, q, s)
        assert int((s != 0).sum()) == len(at) and bool((q[at].abs().amax(dim=1) == 127).all())


# ------------------------------------------------------------------------------------------- projection
class Linear:
    def __init__(self, M, N, K, epilogue, seed, lo=-127, hi=127):
        g = rng(9, M, N, K, seed)
        self.x, self.W = R.integers(g, M, K, lo, hi).cuda(), R.integers(g, N, K, lo, hi).cuda()
        self.xs = torch.from_numpy(g.uniform(0.01, 0.02, M).astype(np.float32)).cuda()
        self.ws = torch.from_numpy(g.uniform(0.001, 0.002, N).astype(np.float32)).cuda()
        self.res = normal(g, M, N).cuda() if epilogue == "bf16_residual" else None
        self.epilogue = epilogue
        self.y = torch.full((M, N), float("nan"), device="cuda",
                            dtype=torch.float32 if epilogue == "fp32" else torch.bfloat16)

    def want(self):
        return R.linear(self.x, self.xs, self.W, self.ws, self.res, self.epilogue)

    def run(self, plan, stream=None):
        plan.run(self.x, self.xs, self.W, self.ws, self.res, self.y, stream)
        return self.y


def check_linear(M, N, K, epilogue, seed=0, lo=-127, hi=127, static=False):
    c = Linear(M, N, K, epilogue, seed, lo, hi)
    plan = skg.Q8Plan(M, N, K, epilogue, static_weights=static)
    try:
        for _ in range(2):                              # a plan is used again
            c.y.fill_(float("nan"))
            c.run(plan)
            assert R.same_bits(c.y, c.want()), f"{M}x{N}x{K} {epilogue}"
    finally:
        plan.close()


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 96, 127, 128, 129, 192, 193,
                               200, 255, 256, 257, 333, 512, 700])
@pytest.mark.parametrize("N,K,epilogue", [(384, 1024, "fp32"), (129, 1040, "bf16_residual"), (1000, 4112, "bf16")])
def test_linear_batches(M, N, K, epilogue):
    check_linear(M, N, K, epilogue)


@pytest.mark.parametrize("M", [1, 7, 16, 50, 150, 300])
@pytest.mark.parametrize("N,K", [(1, 16), (1, 7168), (2, 48), (127, 112), (128, 128), (255, 144), (257, 2064), (5001, 272),
                                 (640, 16400)])
def test_linear_ragged_sizes(M, N, K):
    for epilogue in ("bf16_residual", "fp32"):
        check_linear(M, N, K, epilogue, static=True)


@pytest.mark.parametrize("M,N,K", [(1, 12288, 7168), (8, 7168, 8192), (16, 7168, 7168), (64, 7168, 16384), (64, 384, 7168),
                                   (500, 4096, 7168), (1024, 7168, 4096)])
def test_linear_decode_layer_sizes(M, N, K):
    check_linear(M, N, K, "bf16_residual", static=True)
    check_linear(M, N, K, "fp32", seed=1)


@pytest.mark.parametrize("M", [1, 16, 64, 130])
@pytest.mark.parametrize("K", [1024, 1040, 2048, 131056])
@pytest.mark.parametrize("xv,wv", [(-128, -128), (127, 127), (-128, 127), (127, -127)])
def test_linear_largest_sums(M, K, xv, wv):
    """Every product at its extreme: sums up to 2^31 - 2^18, exact."""
    N = 130
    x = torch.full((M, K), xv, dtype=torch.int8, device="cuda")
    W = torch.full((N, K), wv, dtype=torch.int8, device="cuda")
    x[0, 0], W[1, K - 1] = 1, 1                          # not all sums alike, some odd
    one = torch.ones(max(M, N), device="cuda")
    y = torch.empty(M, N, dtype=torch.float32, device="cuda")
    plan = skg.Q8Plan(M, N, K, "fp32")
    plan.run(x, one[:M], W, one[:N], None, y)
    sums = x.double() @ W.double().t()
    assert torch.equal(y, sums.float())
    plan.close()


def test_linear_every_sum_is_exact():
    """fp32 scales of 2^-8 keep the low bits of sums near 2^24 visible after removing the leading part."""
    M, N, K = 20, 256, 2048
    g = rng(10)
    x, W = R.integers(g, M, K, 100, 127).cuda(), R.integers(g, N, K, 100, 127).cuda()
    sums = (x.double() @ W.double().t())
    assert float(sums.max()) > 2 ** 24                    # beyond what one fp32 accumulation holds exactly
    one = torch.ones(N, device="cuda")
    y = torch.empty(M, N, dtype=torch.float32, device="cuda")
    plan = skg.Q8Plan(M, N, K, "fp32")
    plan.run(x, one[:M], W, one, None, y)
    assert torch.equal(y, sums.float())
    plan.close()


@pytest.mark.parametrize("M", [3, 40, 300])
def test_linear_scales_that_are_not_finite_stay_in_their_rows(M):
    c = Linear(M, 200, 512, "bf16", 3)
    c.xs[M // 2] = float("nan")
    c.x[M // 2] = 0
    c.ws[7] = float("inf")
    c.x[0] = 0
    plan = skg.Q8Plan(M, 200, 512, "bf16")
    c.run(plan)
    assert R.same_bits(c.y, c.want())
    assert bool(c.y[M // 2].isnan().all()) and bool(c.y[0, 7].isnan())
    assert int(c.y[1 if M // 2 != 1 else 2].isnan().sum()) == 0
    plan.close()


def test_linear_beyond_32_bit_offsets():
    """More than 2^31 outputs."""
    M, N, K = 200_000, 11_000, 16
    g = rng(11)
    x, W = R.integers(g, M, K).cuda(), R.integers(g, N, K).cuda()
    xs, ws = torch.ones(M, device="cuda"), torch.full((N,), 0.5, device="cuda")
    y = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    plan = skg.Q8Plan(M, N, K, "bf16")
    plan.run(x, xs, W, ws, None, y)
    at = torch.tensor([0, 1, 97_612, 195_224, 195_225, 195_226, M - 2, M - 1], device="cuda")
    assert R.same_bits(y[at], R.linear(x[at], xs[at], W, ws, None, "bf16"))
    plan.close()


def test_linear_writes_only_its_output():
    M, N, K = 37, 300, 528
    c = Linear(M, N, K, "bf16", 4)
    guard = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    c.y = guard[1:M + 1]
    plan = skg.Q8Plan(M, N, K, "bf16")
    c.run(plan)
    assert R.same_bits(c.y, c.want())
    assert bool((guard[0] == 7).all()) and bool((guard[M + 1] == 7).all())
    plan.close()


def test_side_stream_and_its_order():
    """Everything on one side stream, each call on what the one before wrote."""
    M, N, K = 24, 512, 1024
    g = rng(12)
    x, gamma = normal(g, M, K).cuda(), normal(g, K).cuda()
    W = R.integers(g, N, K).cuda()
    ws = torch.full((N,), 0.002, device="cuda")
    q, s = rows_out(M, K)
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    plan = skg.Q8Plan(M, N, K, "bf16", static_weights=True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        q.fill_(0)
        side.wait_stream(torch.cuda.current_stream())
        skg.skg_rmsnorm_q8(x, None, gamma, EPS, None, q, s, stream=side)
        plan.run(q, s, W, ws, None, y, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert R.same_bits(y, R.linear(q, s, W, ws, None, "bf16"))
    plan.close()


@pytest.mark.parametrize("M", [1, 12, 64, 200])
def test_graph_capture_of_a_block(M):
    """Norm, projection, gated quantiser and projection with residual, captured once and replayed on new inputs."""
    H, F = 1024, 1536
    g = rng(13, M)
    x = normal(g, M, H).cuda()
    gamma = normal(g, H).cuda()
    W1, W2 = R.integers(g, 2 * F, H).cuda(), R.integers(g, H, F).cuda()
    w1, w2 = torch.full((2 * F,), 1e-3, device="cuda"), torch.full((H,), 1e-3, device="cuda")
    q, s = rows_out(M, H)
    a, sa = rows_out(M, F)
    u = torch.empty(M, 2 * F, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(M, H, dtype=torch.bfloat16, device="cuda")
    p1 = skg.Q8Plan(M, 2 * F, H, "bf16", static_weights=True)
    p2 = skg.Q8Plan(M, H, F, "bf16_residual", static_weights=True)

    def block():
        skg.skg_rmsnorm_q8(x, None, gamma, EPS, None, q, s)
        p1.run(q, s, W1, w1, None, u)
        skg.skg_quantize_q8(u[:, F:], u[:, :F], a, sa)
        p2.run(a, sa, W2, w2, x, y)

    block()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block()
    for k in range(5):
        x.copy_(normal(rng(14, M, k), M, H))
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        v, _ = R.norm_rows(x, None, gamma, EPS)
        R.check_rows(v, q, s, R.row_error(H))
        assert R.same_bits(u, R.linear(q, s, W1, w1, None, "bf16"))
        R.check_rows(R.gated_rows(u[:, F:], u[:, :F]), a, sa, R.row_error(F, u[:, :F]))
        assert R.same_bits(y, R.linear(a, sa, W2, w2, x, "bf16_residual"))
    p1.close()
    p2.close()


def test_binding_refuses_wrong_tensors():
    M, N, K = 4, 64, 64
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    q, s = rows_out(M, K)
    bad = [
        lambda: skg.skg_rmsnorm_q8(x.float(), None, None, EPS, None, q, s),
        lambda: skg.skg_rmsnorm_q8(x, x[:2], None, EPS, None, q, s),
        lambda: skg.skg_rmsnorm_q8(x.t(), None, None, EPS, None, q.t(), s),
        lambda: skg.skg_rmsnorm_q8(x, None, x[0, :8], EPS, None, q, s),
        lambda: skg.skg_rmsnorm_q8(x, None, None, EPS, x, q, s),
        lambda: skg.skg_quantize_q8(x, None, q.short(), s),
        lambda: skg.skg_quantize_q8(x, None, q, s.double()),
        lambda: skg.skg_quantize_q8(x[0], None, q, s),
        lambda: skg.skg_quantize_q8(x[:1].expand(M, K), None, q, s),
        lambda: skg.skg_quantize_q8(x, None, q[:, :32], s),
    ]
    c = Linear(M, N, K, "bf16_residual", 5)
    plan = skg.Q8Plan(M, N, K, "bf16_residual")
    good = [c.x, c.xs, c.W, c.ws, c.res, c.y]
    for i, wrong in enumerate([c.x[:2], c.xs[:2], c.W.t(), c.ws.double(), None, c.y.float()]):
        args = list(good)
        args[i] = wrong
        bad.append(lambda args=args: plan.run(*args))
    for k, call in enumerate(bad):
        with pytest.raises(skg.SkgError) as e:
            call()
        assert e.value.status == skg.SKG_ERR_INVALID_ARG, k
    odd = torch.zeros(M * K + 1, dtype=torch.int8, device="cuda")[1:].view(M, K)
    with pytest.raises(skg.SkgError) as e:
        plan.run(odd, c.xs, c.W, c.ws, c.res, c.y)
    assert e.value.status == skg.SKG_ERR_ALIGNMENT
    plan.run(*good)                                       # and the plan still works
    assert R.same_bits(c.y, c.want())
    plan.close()


# ------------------------------------------------------------------------- every kernel at every shape
SHAPES = [(skg.SKG_Q8_KERNEL_SPLIT, t, k) for t in (32, 64) for k in range(1, 9)] + \
         [(skg.SKG_Q8_KERNEL_WIDE, 128, k) for k in range(1, 5)]


@pytest.mark.parametrize("kind,m_tile,split", SHAPES)
@pytest.mark.parametrize("M,N,K", [(1, 128, 1024), (2, 1000, 2064), (16, 300, 1040), (33, 257, 16400), (64, 130, 4096),
                                   (70, 640, 1152), (200, 384, 3104), (193, 129, 16), (130, 2000, 528), (385, 1000, 2048),
                                   (64, 1024, 16384), (50, 3000, 2064), (20, 260, 1024), (300, 10000, 1280)])
def test_every_launch_shape_gives_the_same_bits(M, N, K, kind, m_tile, split):
    """Both tcgen05 kernels at every tile and split, whatever the plan would choose."""
    c = Linear(M, N, K, "bf16_residual", 6)
    want = c.want()
    plan = skg.Q8Plan(M, N, K, "bf16_residual", static_weights=split % 2 == 0)
    plan.force(kind, m_tile, split)
    d = plan.info()
    assert d["m_tile"] == m_tile and d["kernel_kind"] == kind and d["split_k"] == max(1, min(split, -(-K // 128)))
    for _ in range(3):
        c.y.fill_(float("nan"))
        c.run(plan)
        assert R.same_bits(c.y, want)
    plan.check()
    plan.close()


@pytest.mark.parametrize("epilogue", ["bf16", "bf16_residual", "fp32"])
@pytest.mark.parametrize("M,N", [(40, 512), (40, 514), (64, 1023), (100, 300)])
def test_output_addresses(M, N, epilogue):
    """y, residual and scales at addresses that only their element types allow."""
    K = 1024
    c = Linear(M, N, K, epilogue, 16)
    want = c.want()
    out = torch.full((M * N + 1,), 7.0, dtype=c.y.dtype, device="cuda")
    c.y = out[1:].view(M, N)
    for name in ("xs", "ws"):
        v = getattr(c, name)
        setattr(c, name, torch.cat([v[:1], v])[1:])
    if c.res is not None:
        c.res = torch.cat([c.res.flatten()[:1], c.res.flatten()])[1:].view(M, N)
    plan = skg.Q8Plan(M, N, K, epilogue)
    c.run(plan)
    assert R.same_bits(c.y, want) and out[0] == 7
    plan.close()


@pytest.mark.parametrize("M", [1, 5, 8, 9, 16])
@pytest.mark.parametrize("N", [1, 77, 2432, 2433, 4864, 5000, 7296, 7297, 12288])
@pytest.mark.parametrize("K", [16, 1040, 4112])
def test_streaming_kernel_at_every_launch_shape(M, N, K):
    c = Linear(M, N, K, "bf16_residual", 7)
    plan = skg.Q8Plan(M, N, K, "bf16_residual", static_weights=(N + K) % 2 == 0)
    plan.force(skg.SKG_Q8_KERNEL_STREAM)
    assert R.same_bits(c.run(plan), c.want())
    plan.close()


def test_streaming_kernel_refuses_more_tokens():
    plan = skg.Q8Plan(17, 128, 128, "bf16")
    with pytest.raises(skg.SkgError) as e:
        plan.force(skg.SKG_Q8_KERNEL_STREAM)
    assert e.value.status == skg.SKG_ERR_UNSUPPORTED and plan.info()["kernel"] == "q8_split"
    plan.close()


@pytest.mark.parametrize("kind,m_tile,split", SHAPES[::3])
@pytest.mark.parametrize("v", [(-128, -128), (127, -128)])
def test_largest_sums_on_every_launch_shape(kind, m_tile, split, v):
    M, N, K = 20, 130, 131056
    x = torch.full((M, K), v[0], dtype=torch.int8, device="cuda")
    W = torch.full((N, K), v[1], dtype=torch.int8, device="cuda")
    x[0, 0], W[1, K - 1] = 1, 1
    one = torch.ones(N, device="cuda")
    y = torch.empty(M, N, dtype=torch.float32, device="cuda")
    plan = skg.Q8Plan(M, N, K, "fp32")
    plan.force(kind, m_tile, split)
    plan.run(x, one[:M], W, one, None, y)
    assert torch.equal(y, (x.double() @ W.double().t()).float())
    plan.close()


def test_plans_share_no_state_between_streams():
    """Two plans of one shape on two streams at once."""
    M, N, K = 48, 2000, 4096
    cs = [Linear(M, N, K, "fp32", 20 + i) for i in range(2)]
    plans = [skg.Q8Plan(M, N, K, "fp32", static_weights=True) for _ in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    want = [c.want() for c in cs]
    torch.cuda.synchronize()
    for _ in range(30):
        for c, p, s in zip(cs, plans, streams):
            c.run(p, s)
    for c, p, w in zip(cs, plans, want):
        p.check()
        assert R.same_bits(c.y, w)
        p.close()


def test_bounded_wait_is_reported_and_the_plan_recovers():
    c = Linear(24, 500, 4096, "fp32", 8)
    plan = skg.Q8Plan(24, 500, 4096, "fp32")
    want = c.want()
    skg.skg_q8_debug_wait_timeout(plan.handle, 2_000_000)
    with pytest.raises(skg.SkgError) as e:
        plan.check()
    assert e.value.status == skg.SKG_ERR_DEVICE_TIMEOUT
    plan.check()
    skg.skg_q8_debug_wait_timeout(plan.handle, 1_000_000)
    torch.cuda.synchronize()
    with pytest.raises(skg.SkgError) as e:
        c.run(plan)
    assert e.value.status == skg.SKG_ERR_DEVICE_TIMEOUT
    c.run(plan)
    assert R.same_bits(c.y, want)
    plan.check()
    plan.close()


@pytest.mark.parametrize("M", [1, 20, 100])
def test_mlp_block(M):
    """The block of q8_block.py, each stage from what the one before left."""
    from projection_gemm_gb300.q8_block import Q8MLP
    H, F, E = 512, 768, 48
    g = rng(15, M)
    x, r, gamma = normal(g, M, H).cuda(), normal(g, M, H).cuda(), (normal(g, H, std=0.2) + 1).cuda()
    W1, W2 = normal(g, 2 * F, H, std=H ** -0.5).cuda(), normal(g, H, F, std=F ** -0.5).cuda()
    Wr = normal(g, E, H, std=H ** -0.5).cuda() if M <= 64 else None
    b = Q8MLP(M, gamma, W1, W2, Wr)
    R.check_rows(W1.double(), b.gate_up, b.gate_up_scale, R.row_error(H))
    R.check_rows(W2.double(), b.down, b.down_scale, R.row_error(F))
    out, scores = b.run(x, r)
    b.check()
    v, _ = R.norm_rows(x, r, gamma, 1e-6)
    R.check_rows(v, b.q, b.scale, R.row_error(H))
    assert torch.equal(b.h, (x.float() + r.float()).to(torch.bfloat16))
    assert R.same_bits(b.u, R.linear(b.q, b.scale, b.gate_up, b.gate_up_scale, None, "bf16"))
    R.check_rows(R.gated_rows(b.u[:, F:], b.u[:, :F]), b.a, b.a_scale, R.row_error(F, b.u[:, :F]))
    assert R.same_bits(out, R.linear(b.a, b.a_scale, b.down, b.down_scale, b.h, "bf16_residual"))
    if Wr is not None:
        want = b.v.double() @ Wr.double().t()
        s1 = b.v.double().abs() @ Wr.double().abs().t()
        assert bool(((scores.double() - want).abs() <= 2.0 ** -16 * s1 + 2.0 ** -23 * want.abs()).all())
    # And the whole against the unquantised block.  Rounding to a step of max / 127 is off by step / sqrt(12):
    # for normal rows (max 4 rms) 0.9% of the rms, for a's (products of two, max 12 rms) 2.7%.  W1 and v give u
    # 1.3%, which enters a about twice; with a's and W2's own that is 3.4%; half as much again is allowed.
    u = (v @ W1.double().t())
    ref = (u[:, F:] * u[:, :F] / (1 + torch.exp(-u[:, :F]))) @ W2.double().t()
    off = (out.double() - (x.double() + r.double()) - ref).norm() / ref.norm()
    assert float(off) < 0.05
    b.close()
