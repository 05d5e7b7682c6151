"""The 8-bit path where a bound leaves room: integers that have to be equal,
values at the ends of their types' ranges, and sizes at the ends of theirs."""
import numpy as np
import pytest
import torch

from projection_gemm_gb300 import skg
from tests import q8_reference as R
from tests.test_q8_gpu import Linear, normal, rng, rows_out


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


# ------------------------------------------------------------------------------------------------- norm
LENGTHS = [8, 256, 1000, 1024, 5001, 7168, 16384, 20001]          # every form of the row kernels


def check_norm(x, residual, gamma, eps):
    eps = float(np.float32(eps))
    M, K = x.shape
    q, s = rows_out(M, K)
    y = torch.empty_like(x)
    skg.skg_rmsnorm_q8(x, residual, gamma, eps, None, q, s, y)
    v, _ = R.norm_rows(x, residual, gamma, eps)
    e = R.row_error(K)
    R.check_rows(v, q, s, e, f"{M}x{K} eps={eps}")
    assert bool(((y.double() - v).abs() <= (2.0 ** -8 + e) * v.abs() + 2.0 ** -133).all())


@pytest.mark.gpu
@pytest.mark.parametrize("K", LENGTHS)
@pytest.mark.parametrize("eps", [0.0, 1e-6, 3e38])
def test_norm_of_the_largest_values(K, eps):
    """The sum of squares leaves fp32's range, by up to K 2^128; one small value among them stays what it is."""
    g = rng(31, K)
    x = torch.from_numpy(g.choice([-1.0, 1.0], size=(5, K))).float() * 3.38e38
    x[1] *= torch.from_numpy(g.uniform(0, 1, K)).float()
    x[2] *= 1e-17
    x[3] *= 2.0 ** -20
    x[4, 1:] = 1e-30
    x = x.to(torch.bfloat16).cuda()
    check_norm(x, None, (normal(g, K, std=0.2) + 1).cuda(), eps)
    check_norm(x[2:], normal(g, 3, K).cuda(), None, eps)


@pytest.mark.gpu
@pytest.mark.parametrize("K", LENGTHS)
@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-36, 1e-30])
def test_norm_of_the_smallest_values(K, eps):
    """Squares below fp32's range, which eps does not cover."""
    g = rng(32, K)
    sizes = [1e-8, 1e-15, 1e-18, 1e-20, 1e-21, 1e-22, 5e-23, 1e-23, 1e-30, 1e-37, 1e-39]
    x = torch.stack([normal(g, K).float() * v for v in sizes]).to(torch.bfloat16)
    x[:, 0] = torch.tensor(sizes).to(torch.bfloat16)
    x[-1, 1:] = 0                                       # one value alone
    x = x.cuda()
    check_norm(x, None, (normal(g, K, std=0.2) + 1).cuda(), eps)
    check_norm(x, x.flip(0).contiguous(), None, eps)


@pytest.mark.gpu
@pytest.mark.parametrize("K", [8, 1001, 20001])
def test_norm_of_zeros(K):
    """0 with eps; 0 / 0 without."""
    x = torch.zeros(2, K, dtype=torch.bfloat16, device="cuda")
    for eps in (1e-6, 0.0):
        q, s = rows_out(2, K)
        skg.skg_rmsnorm_q8(x, None, None, eps, None, q, s)
        assert bool((q == 0).all()) and bool((s == 0).all() if eps else s.isnan().all())


@pytest.mark.gpu
@pytest.mark.parametrize("K", LENGTHS)
@pytest.mark.parametrize("lo,hi,size", [(-104, -88, 1e2), (-120, -100, 1e20), (-200, -150, 3e38), (-130, -86, 1e30)])
def test_quantize_rows_of_large_negative_gates(K, lo, hi, size):
    """exp(g) below fp32's range, its product with x within: the row has the values of the formula."""
    g = rng(33, K, -lo)
    gate = torch.from_numpy(g.uniform(lo, hi, size=(6, K))).to(torch.bfloat16).cuda()
    x = torch.from_numpy(g.uniform(0.25, 1, size=(6, K)) * size * g.choice([-1.0, 1.0], size=(6, K))).to(torch.bfloat16).cuda()
    v = R.gated_rows(x, gate)
    q, s = rows_out(6, K)
    skg.skg_quantize_q8(x, gate, q, s)
    R.check_rows(v, q, s, R.row_error(K, gate))


# -------------------------------------------------------------------------------- the ends of the sizes
LARGEST = 2 ** 31 - 1


@pytest.mark.gpu
def test_the_longest_row():
    x = torch.zeros(1, LARGEST, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1023, 1024, 2 ** 30, LARGEST - 1025, LARGEST - 1024, LARGEST - 1], device="cuda")
    x[0, at] = normal(rng(34), len(at)).cuda()
    q, s = rows_out(1, LARGEST)
    skg.skg_quantize_q8(x, None, q, s)
    want, _ = nearest_even(x[:, at])
    assert torch.equal(q[:, at].long(), want) and int(torch.count_nonzero(q)) == int((want != 0).sum())
    assert s[0] == (x[:, at].abs().amax().double() / 127).float()


@pytest.mark.gpu
def test_the_most_rows():
    """One element each: its integer is -127, 0 or 127."""
    x = torch.zeros(LARGEST, 1, dtype=torch.bfloat16, device="cuda")
    x[::3] = 2.0
    x[1::3] = -0.5
    x[LARGEST - 1] = 3.0
    q, s = rows_out(LARGEST, 1)
    skg.skg_quantize_q8(x, None, q, s)
    assert q[LARGEST - 1].item() == 127 and s[LARGEST - 1] == torch.tensor(3.0) / 127
    for first, integer, size in ((0, 127, 2.0), (1, -127, 0.5), (2, 0, 0.0)):
        end = LARGEST - 1
        assert bool((q[first:end:3] == integer).all()) and bool((s[first:end:3] == torch.tensor(size) / 127).all())


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 8])
def test_the_most_channels(M):
    N, K = LARGEST, 16
    W = torch.randint(-128, 128, (N, K), dtype=torch.int8, device="cuda", generator=torch.Generator("cuda").manual_seed(35))
    x, xs = R.integers(rng(35), M, K).cuda(), torch.full((M,), 0.5, device="cuda")
    ws = torch.ones(N, device="cuda")
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    plan = skg.Q8Plan(M, N, K, "bf16", static_weights=True)
    plan.run(x, xs, W, ws, None, y)
    for a in range(0, N, N // 7):
        b = min(a + 1_000_000, N)
        assert R.same_bits(y[:, a:b], R.linear(x, xs, W[a:b], ws[a:b], None, "bf16"))
    assert R.same_bits(y[:, N - 1000:], R.linear(x, xs, W[N - 1000:], ws[N - 1000:], None, "bf16"))
    assert not bool(y.isnan().any())
    plan.close()


@pytest.mark.parametrize("call", [
    lambda v: skg.skg_q8_plan_query(v, 128, 128, "bf16", 152), lambda v: skg.skg_q8_plan_query(4, v, 128, "bf16", 152),
    lambda v: skg.skg_q8_plan_query(4, 128, v, "bf16", 152), lambda v: skg.skg_q8_plan_query(4, 128, 128, v, 152),
    lambda v: skg.skg_q8_plan_query(4, 128, 128, "bf16", v), lambda v: skg.skg_q8_plan(v, 128, 128, "bf16"),
    lambda v: skg.skg_q8_plan(4, v, 128, "bf16"), lambda v: skg.skg_q8_plan(4, 128, v, "bf16"),
    lambda v: skg.skg_q8_plan_force(None, v), lambda v: skg.skg_q8_plan_force(None, 0, 0, v)])
def test_sizes_beyond_32_bits_are_refused_not_cut(call):
    for v in (2 ** 32 + 16, 2 ** 33 + 128, 2 ** 31, -2 ** 32 + 16):
        with pytest.raises(skg.SkgError) as e:
            call(v)
        assert e.value.status == skg.SKG_ERR_INVALID_ARG


@pytest.mark.parametrize("shape", [(2 ** 32 + 5, 1), (1, 2 ** 32 + 8), (2 ** 31, 1)])
def test_rows_beyond_32_bits_are_refused_not_cut(shape):
    """A tensor as the binding sees one: shape, type, strides, place."""
    class Huge:
        dtype, is_cuda = torch.bfloat16, True

        def __init__(self, shape, dtype=torch.bfloat16):
            self.shape, self.dtype = torch.Size(shape), dtype

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return 1 << 20

        def get_device(self):
            return 0

    x, q, s = Huge(shape), Huge(shape, torch.int8), Huge(shape[:1], torch.float32)
    for call in (lambda: skg.skg_rmsnorm_q8(x, None, None, 1e-6, None, q, s, stream=0),
                 lambda: skg.skg_quantize_q8(x, None, q, s, stream=0)):
        with pytest.raises(skg.SkgError) as e:
            call()
        assert e.value.status == skg.SKG_ERR_INVALID_ARG


# ------------------------------------------------------------------------------------------- projection
def cancelling(g, M, N, K):
    """Operands whose sums over the first half of K are near 127^2 K / 2 and over all of it small: what an addition
    of large partial sums loses shows in every bit of the result."""
    half = K // 2
    x, W = R.integers(g, M, K, 100, 127), R.integers(g, N, K, 100, 127)
    x[:, half:] = x[:, :half]
    W[:, half:] = -W[:, :half]
    at = torch.from_numpy(g.choice(K, size=40, replace=False))
    x[:, at] = R.integers(g, M, 40)
    W[:, at] = R.integers(g, N, 40)
    return x.cuda(), W.cuda()


STREAM = (skg.SKG_Q8_KERNEL_STREAM, 0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("kind,m_tile,split", [STREAM] + [(skg.SKG_Q8_KERNEL_SPLIT, t, k) for t in (32, 64) for k in range(1, 9)] +
                         [(skg.SKG_Q8_KERNEL_WIDE, 128, k) for k in range(1, 5)])
def test_large_partial_sums_that_cancel(kind, m_tile, split):
    for M, N, K in [(16, 260, 16400), (70, 130, 8192)]:
        if kind == skg.SKG_Q8_KERNEL_STREAM and M > 16:
            continue
        x, W = cancelling(rng(36, M, K), M, N, K)
        sums = x.double() @ W.double().t()
        half = (x[:, :K // 2].double() @ W[:, :K // 2].double().t()).abs().max()
        assert float(half) > 2 ** 25 and float(sums.abs().max()) < 2 ** 24
        one = torch.ones(max(M, N), device="cuda")
        y = torch.empty(M, N, dtype=torch.float32, device="cuda")
        plan = skg.Q8Plan(M, N, K, "fp32")
        plan.force(kind, m_tile, split)
        plan.run(x, one[:M], W, one[:N], None, y)
        assert torch.equal(y.double(), sums)
        plan.close()


def with_workspace(M, N, K):
    """A plan that puts sums away: K of one CTA."""
    plan = skg.Q8Plan(M, N, K, "fp32", static_weights=True)
    plan.force(skg.SKG_Q8_KERNEL_SPLIT, 64 if M > 32 else 32, 1)
    assert plan.info()["workspace_bytes"] > 0
    return plan


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(48, 2000, 8192), (20, 300, 16400), (200, 640, 5120)])
def test_workspaces_of_two_plans_at_once(M, N, K):
    cs = [Linear(M, N, K, "fp32", 40 + i) for i in range(2)]
    plans, streams = [with_workspace(M, N, K) for _ in cs], [torch.cuda.Stream() for _ in cs]
    want = [c.want() for c in cs]
    torch.cuda.synchronize()
    for _ in range(30):
        for c, p, s in zip(cs, plans, streams):
            c.run(p, s)
    for c, p, w in zip(cs, plans, want):
        p.check()
        assert R.same_bits(c.y, w)
        p.close()


@pytest.mark.gpu
@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("M,N,K", [(48, 2000, 8192), (20, 300, 16400), (64, 7168, 7168), (200, 640, 5120)])
def test_runs_of_one_plan_follow_each_other_with_nothing_between(M, N, K, graph):
    """Alternating inputs, an output each: a run's sums in the workspace are not the next one's."""
    cs = [Linear(M, N, K, "fp32", 50 + i) for i in range(2)]
    want = [c.want() for c in cs]
    ys = [torch.full((M, N), float("nan"), device="cuda") for _ in range(12)]
    plan = with_workspace(M, N, K)

    def runs():
        for i, y in enumerate(ys):
            c = cs[i % 2]
            plan.run(c.x, c.xs, c.W, c.ws, None, y)

    torch.cuda.synchronize()
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            runs()
        g.replay()
    else:
        runs()
    plan.check()
    torch.cuda.synchronize()
    for i, y in enumerate(ys):
        assert R.same_bits(y, want[i % 2]), i
    plan.close()


@pytest.mark.gpu
def test_a_graph_of_a_plan_forced_to_other_workspaces():
    """Runs captured with a workspace that the plan then outgrows keep their own."""
    M, N, K = 40, 640, 16384
    c = Linear(M, N, K, "fp32", 60)
    want = c.want()
    plan = skg.Q8Plan(M, N, K, "fp32")
    graphs = []
    for split in (8, 4, 2, 1):
        plan.force(skg.SKG_Q8_KERNEL_SPLIT, 64, split)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(plan)
        graphs.append(g)
    assert plan.info()["workspace_bytes"] > 0
    for g in graphs + graphs[::-1]:
        c.y.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert R.same_bits(c.y, want)
    plan.close()


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(300, 10000, 1280), (130, 2000, 528), (1500, 2300, 2064), (129, 257, 128), (4096, 3000, 384)])
def test_wide_runs_follow_each_other_with_nothing_between(M, N, K):
    """The widened operands of one launch's last units and of the next one's first."""
    cs = [Linear(M, N, K, "fp32", 70 + i) for i in range(2)]
    want = [c.want() for c in cs]
    ys = [torch.full((M, N), float("nan"), device="cuda") for _ in range(10)]
    for split in (1, 2):
        plan = skg.Q8Plan(M, N, K, "fp32", static_weights=split == 1)
        plan.force(skg.SKG_Q8_KERNEL_WIDE, 128, split)
        torch.cuda.synchronize()
        for _ in range(3):
            for i, y in enumerate(ys):
                c = cs[i % 2]
                plan.run(c.x, c.xs, c.W, c.ws, None, y)
        plan.check()
        for i, y in enumerate(ys):
            assert R.same_bits(y, want[i % 2]), (split, i)
        plan.close()


@pytest.mark.gpu
@pytest.mark.parametrize("M", [20, 200])
def test_a_projection_after_a_kernel_that_takes_long(M):
    """The bounded waits of a launch that starts early do not count what the kernel before it takes."""
    x = torch.zeros(1, LARGEST, dtype=torch.bfloat16, device="cuda")
    x[0, -1] = 2.0 ** -90                               # with eps = 0 the sum is taken twice: longer than the limit
    h, y = torch.empty_like(x), torch.empty_like(x)
    q, s = rows_out(1, LARGEST)
    c = Linear(M, 500, 1024, "bf16", 80)
    want = c.want()
    plan = skg.Q8Plan(M, 500, 1024, "bf16", static_weights=True)
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    a.record()
    skg.skg_rmsnorm_q8(x, x, x[0], 0.0, h, q, s, y)
    c.run(plan)
    b.record()
    plan.check()
    assert R.same_bits(c.y, want) and q[0, -1] == 127
    assert a.elapsed_time(b) > 1000
    plan.close()
