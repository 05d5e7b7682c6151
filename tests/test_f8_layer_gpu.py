"""The 8-bit floating point path's and the experts' operators together on a GB300:
a layer of experts stage by stage, in graphs, on several streams, back to back, and
what a plan reports."""
import pytest
import torch

from projection_gemm_gb300 import skg
from projection_gemm_gb300.f8_experts import F8Experts, main
from tests import f8_reference as R
from tests.test_experts_gpu import U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from projection_gemm_gb300 import build
    build.build()
    skg.load()
    assert torch.cuda.is_available()


def normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16).cuda()


def make(T, k, E, hidden, inner, seed=1, dropped=0.0, router=False):
    g = torch.Generator().manual_seed(seed)
    W1, W2 = normal(g, E, 2 * inner, hidden, std=hidden ** -0.5), normal(g, E, hidden, inner, std=inner ** -0.5)
    layer = F8Experts(T, k, W1, W2, normal(g, E, hidden) if router else None)
    return layer, choices(g, T, k, E, hidden, dropped)


def choices(g, T, k, E, hidden, dropped=0.0):
    expert = torch.topk(torch.randn(T, E, generator=g), k, 1).indices.int()
    expert[torch.rand(T, k, generator=g) < dropped] = -1
    return normal(g, T, hidden), normal(g, T, hidden), expert.cuda(), torch.rand(T, k, generator=g).cuda()


@pytest.mark.parametrize("T,k,E,hidden,inner,dropped", [(1, 2, 4, 256, 128, 0.0), (37, 3, 12, 400, 272, 0.2),
                                                        (64, 8, 64, 1024, 256, 0.0), (700, 4, 6, 512, 640, 0.1), (5, 2, 3, 144, 48, 1.0)])
def test_layer_stage_by_stage(T, k, E, hidden, inner, dropped):
    layer, (x, res, expert, weight) = make(T, k, E, hidden, inner, dropped=dropped)
    out = layer.run(x, res, expert, weight)
    layer.check()
    at = layer.offsets.tolist()
    n = at[-1]
    assert n == int((expert >= 0).sum())
    rows = layer.rows[:n].long()
    if n:
        R.check_quantised(x[rows], layer.q[:n], layer.q_scale[:n])
        R.check_gated(layer.u[:n, inner:], layer.u[:n, :inner], layer.a[:n], layer.a_scale[:n])
    for e in range(E):
        s = slice(at[e], at[e + 1])
        if s.stop > s.start:
            R.check_linear(layer.q[s], layer.q_scale[s], layer.gate_up[e], layer.gate_up_scale[e], None, layer.u[s])
            R.check_linear(layer.a[s], layer.a_scale[s], layer.down[e], layer.down_scale[e], None, layer.d[s])
    live = layer.pos >= 0
    terms = torch.where(live[..., None], layer.d[layer.pos.clamp(min=0).long()].double(), 0.0) * weight.double()[..., None]
    want, mass = res.double() + terms.sum(1), res.double().abs() + terms.abs().sum(1)
    assert bool(((out.double() - want).abs() <= (k + 1) * U * mass * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()).all())
    layer.close()


@pytest.mark.parametrize("T,k,E", [(4, 2, 16), (300, 4, 5)])
def test_layer_in_a_graph_with_other_inputs(T, k, E):
    """Captured once on a stream of its own, replayed for other tokens and choices (also none at all): the bits of the
    eager step."""
    hidden, inner = 512, 256
    layer, _ = make(T, k, E, hidden, inner)
    g = torch.Generator().manual_seed(7)
    inputs = [choices(g, T, k, E, hidden, d) for d in (0.0, 0.5, 1.0, 0.0)]
    want = [layer.run(*i).clone() for i in inputs]
    held = [t.clone() for t in inputs[0]]
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        layer.run(*held)
    for _ in range(3):
        for i, w in zip(inputs, want):
            for h, t in zip(held, i):
                h.copy_(t)
            graph.replay()
            assert torch.equal(layer.out, w)
    layer.check()
    layer.close()


def test_one_plan_in_several_streams_and_graphs_at_once():
    g = torch.Generator().manual_seed(3)
    M, N, K, E = 96, 640, 1024, 6
    W = (torch.randn(E, N, K, generator=g) * 100).clamp(-448, 448).to(R.F8).cuda()
    ws = torch.rand(E, 5, 8, generator=g).cuda()
    plan = skg.F8Plan(M, N, K, "bf16", experts=E)
    jobs = []
    for i in range(4):
        x = (torch.randn(M, K, generator=g) * 100).clamp(-448, 448).to(R.F8).cuda()
        xs = torch.rand(M, 8, generator=g).cuda()
        cuts = torch.sort(torch.randint(0, M + 1, (E - 1,), generator=g)).values.int()
        offsets = torch.cat([torch.zeros(1, dtype=torch.int32), cuts, torch.full((1,), M, dtype=torch.int32)]).cuda()
        y = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
        plan.run(x, xs, W, ws, None, y, offsets=offsets)
        jobs.append((x, xs, offsets, y.clone(), y, torch.cuda.Stream()))
    torch.cuda.synchronize()
    graphs = []
    for x, xs, offsets, want, y, s in jobs[2:]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            plan.run(x, xs, W, ws, None, y, offsets=offsets)
        graphs.append(graph)
    for _ in range(20):
        for x, xs, offsets, want, y, s in jobs:
            y.zero_()
        torch.cuda.synchronize()
        for x, xs, offsets, want, y, s in jobs[:2]:
            plan.run(x, xs, W, ws, None, y, offsets=offsets, stream=s)
        for graph, job in zip(graphs, jobs[2:]):
            with torch.cuda.stream(job[5]):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, want) for _, _, _, want, y, _ in jobs)
    plan.check()


@pytest.mark.parametrize("M,N,K,launch", [(1, 2048, 2048, None), (16, 512, 4096, (1, 16, 8)), (64, 1024, 1024, (1, 64, 1)),
                                          (200, 1024, 1024, (2, 128, 2)), (300, 1024, 1024, (2, 256, 1))])
def test_chain_reads_what_the_kernel_before_wrote(M, N, K, launch):
    """Quantiser and projection in turn, each early by programmatic launch, weights static: 200 links without a
    synchronisation, each from a different scale of x, against the same links one at a time."""
    g = torch.Generator().manual_seed(5)
    x = normal(g, M, K)
    W = (torch.randn(N, K, generator=g) * 100).clamp(-448, 448).to(R.F8).cuda()
    ws = torch.rand(R.blocks(N), R.blocks(K), generator=g).cuda()
    plan = skg.F8Plan(M, N, K, "bf16", static_weights=True)
    if launch:
        plan.force(*launch)
    inputs = [x * (2.0 ** (i % 5)) * (1 - 2 * (i % 2)) for i in range(8)]
    q, s = torch.empty(M, K, device="cuda").to(R.F8), torch.empty(M, R.blocks(K), device="cuda")
    ys = [torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(200)]
    want = []
    for v in inputs:
        skg.skg_quantize_f8(v, None, q, s)
        torch.cuda.synchronize()
        plan.run(q, s, W, ws, None, ys[0])
        torch.cuda.synchronize()
        want.append(ys[0].clone())
    for i, y in enumerate(ys):
        skg.skg_quantize_f8(inputs[i % 8], None, q, s)
        plan.run(q, s, W, ws, None, y)
    torch.cuda.synchronize()
    plan.check()
    assert all(torch.equal(y, want[i % 8]) for i, y in enumerate(ys))


@pytest.mark.parametrize("launch", [(1, 16, 3), (1, 64, 1), (2, 128, 1), (2, 256, 2)])
def test_a_row_does_not_depend_on_the_others(launch):
    g = torch.Generator().manual_seed(6)
    M, N, K = 290, 384, 1040
    x = (torch.randn(M, K, generator=g) * 100).clamp(-448, 448).to(R.F8).cuda()
    W = (torch.randn(N, K, generator=g) * 100).clamp(-448, 448).to(R.F8).cuda()
    xs, ws = torch.rand(M, 9, generator=g).cuda(), torch.rand(3, 9, generator=g).cuda()

    def run(order):
        y = torch.empty(len(order), N, device="cuda")
        plan = skg.F8Plan(len(order), N, K, "fp32")
        plan.force(*launch)
        plan.run(x[order].contiguous(), xs[order].contiguous(), W, ws, None, y)
        plan.check()
        return y

    whole = run(torch.arange(M, device="cuda"))
    order = torch.randperm(M, generator=g).cuda()
    assert torch.equal(run(order), whole[order])
    assert torch.equal(run(order[:7]), whole[order[:7]])
    again = run(torch.arange(M, device="cuda"))
    assert torch.equal(again, whole)


def test_a_wait_that_runs_out_is_reported_once():
    plan = skg.F8Plan(2, 128, 128, "bf16")
    skg.skg_f8_debug_wait_timeout(plan.handle, 1000000)
    with pytest.raises(skg.SkgError) as e:
        plan.check()
    assert e.value.status == skg.SKG_ERR_DEVICE_TIMEOUT
    plan.check()
    skg.skg_f8_debug_wait_timeout(plan.handle, 1000000)
    torch.cuda.synchronize()
    x, xs = torch.zeros(2, 128, device="cuda").to(R.F8), torch.zeros(2, 1, device="cuda")
    W, ws = torch.zeros(128, 128, device="cuda").to(R.F8), torch.zeros(1, 1, device="cuda")
    y = torch.empty(2, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(skg.SkgError) as e:
        plan.run(x, xs, W, ws, None, y)
    assert e.value.status == skg.SKG_ERR_DEVICE_TIMEOUT
    plan.run(x, xs, W, ws, None, y)
    plan.check()
    assert bool((y == 0).all())


def test_run_refuses_what_does_not_belong_to_the_plan():
    E, M, N, K = 3, 8, 128, 256
    x, xs = torch.zeros(M, K, device="cuda").to(R.F8), torch.zeros(M, 2, device="cuda")
    W, ws = torch.zeros(E, N, K, device="cuda").to(R.F8), torch.zeros(E, 1, 2, device="cuda")
    y, off = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda"), torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    one, some = skg.F8Plan(M, N, K, "bf16"), skg.F8Plan(M, N, K, "bf16", experts=E)
    res = skg.F8Plan(M, N, K, "bf16_residual")
    bad = [
        lambda: one.run(x, xs, W[0], ws[0], None, y, offsets=off), lambda: some.run(x, xs, W, ws, None, y),
        lambda: one.run(x, xs, W[0], ws[0], y, y), lambda: res.run(x, xs, W[0], ws[0], None, y),
        lambda: one.run(x, xs[:, :1].contiguous(), W[0], ws[0], None, y), lambda: one.run(x, xs, W, ws, None, y),
        lambda: some.run(x, xs, W, ws, None, y, offsets=off[:3].contiguous()),
        lambda: some.run(x, xs, W, ws, None, y, offsets=off.long()),
        lambda: one.run(x.float(), xs, W[0], ws[0], None, y), lambda: one.run(x, xs, W[0], ws[0], None, y.float()),
        lambda: one.run(x.t().contiguous().t(), xs, W[0], ws[0], None, y),
    ]
    for call in bad:
        with pytest.raises(skg.SkgError) as e:
            call()
        assert e.value.status == skg.SKG_ERR_INVALID_ARG
    with pytest.raises(skg.SkgError) as e:                  # a slice that is not 16-byte aligned
        buf = torch.zeros(M * K + 8, device="cuda").to(R.F8)
        one.run(buf[8:].view(M, K), xs, W[0], ws[0], None, y)
    assert e.value.status == skg.SKG_ERR_ALIGNMENT
    for kw, status in ((dict(kind=3), skg.SKG_ERR_INVALID_ARG), (dict(kind=1, m_tile=128), skg.SKG_ERR_INVALID_ARG),
                       (dict(kind=2, m_tile=64), skg.SKG_ERR_INVALID_ARG), (dict(kind=1, split_k=9), skg.SKG_ERR_INVALID_ARG),
                       (dict(kind=2, split_k=5), skg.SKG_ERR_INVALID_ARG), (dict(split_k=-1), skg.SKG_ERR_INVALID_ARG)):
        with pytest.raises(skg.SkgError) as e:
            one.force(**kw)
        assert e.value.status == status


@pytest.mark.parametrize("M,N,K,epilogue,launch", [
    (3, 130, 256, "bf16", (1, 16, 2)), (40, 129, 400, "bf16_residual", (2, 128, 1)), (300, 136, 272, "fp32", (2, 256, 1)),
    (300, 136, 272, "bf16", (2, 256, 2)), (70, 200, 144, "bf16", (1, 64, 1))])
def test_outputs_of_any_alignment_and_nothing_beyond_them(M, N, K, epilogue, launch):
    """y and residual inside larger tensors, one element off: the results of aligned ones, and their neighbours stay."""
    g = torch.Generator().manual_seed(M + N)
    x = (torch.randn(M, K, generator=g) * 100).clamp(-448, 448).to(R.F8).cuda()
    W = (torch.randn(N, K, generator=g) * 100).clamp(-448, 448).to(R.F8).cuda()
    xs, ws = torch.rand(M, R.blocks(K), generator=g).cuda(), torch.rand(R.blocks(N), R.blocks(K), generator=g).cuda()
    dtype = torch.float32 if epilogue == "fp32" else torch.bfloat16
    plan = skg.F8Plan(M, N, K, epilogue)
    plan.force(*launch)

    def run(off):
        big = torch.full((M * N + 64,), 3.0, dtype=dtype, device="cuda")
        y = big[off:off + M * N].view(M, N)
        r = None
        if epilogue == "bf16_residual":
            held = torch.zeros(M * N + off, dtype=torch.bfloat16, device="cuda")
            held[off:] = torch.ones(M * N, dtype=torch.bfloat16, device="cuda")
            r = held[off:].view(M, N)
        plan.run(x, xs, W, ws, r, y)
        plan.check()
        assert bool((big[:off] == 3).all()) and bool((big[off + M * N:] == 3).all())
        return y.clone()

    first = run(0)
    for off in (1, 2, 4, 7):
        assert torch.equal(run(off), first)


def test_example_runs(capsys):
    main(["4", "256", "128", "8", "2"])
    main(["100", "512", "256", "6", "3"])
    assert capsys.readouterr().out.count("unquantised") == 2


@pytest.mark.parametrize("launch", [(1, 16, 1), (1, 32, 4), (1, 64, 1), (2, 128, 2), (2, 256, 1)])
def test_nan_numbers_stay_in_their_row_and_channel(launch):
    g = torch.Generator().manual_seed(8)
    M, N, K = 50, 260, 272
    x = (torch.randn(M, K, generator=g) * 100).clamp(-448, 448)
    W = (torch.randn(N, K, generator=g) * 100).clamp(-448, 448)
    x[7, 200], x[20, 0], W[130, 271], W[259, 5] = (float("nan"),) * 4
    xs, ws = torch.rand(M, 3, generator=g).cuda(), torch.rand(3, 3, generator=g).cuda()
    y = torch.empty(M, N, device="cuda")
    plan = skg.F8Plan(M, N, K, "fp32")
    plan.force(*launch)
    plan.run(x.to(R.F8).cuda(), xs, W.to(R.F8).cuda(), ws, None, y)
    plan.check()
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[[7, 20]] = True
    bad[:, [130, 259]] = True
    assert torch.equal(y.isnan().cpu(), bad)


# ------------------------------------------------------------------------------ beyond 2^31 elements
def test_quantiser_and_rows_beyond_31_bits():
    N, T = 7168, 4096
    M = 2 ** 31 // N + 700
    g = torch.Generator().manual_seed(9)
    x = normal(g, T, N)
    rows = (torch.arange(M, device="cuda", dtype=torch.int32) * 5) % T
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    skg.skg_experts_gather(x, rows, out)
    for s in (slice(0, 64), slice(M - 600, M)):
        assert torch.equal(out[s], x[rows[s].long()])
    q, scale = torch.empty(M, N, dtype=R.F8, device="cuda"), torch.empty(M, 56, device="cuda")
    skg.skg_quantize_f8(out, None, q, scale)
    R.check_quantised(out[M - 600:], q[M - 600:], scale[M - 600:])
    pos = torch.arange(M - 64, M, device="cuda", dtype=torch.int32).view(16, 4)
    back = torch.empty(16, N, dtype=torch.bfloat16, device="cuda")
    skg.skg_experts_combine(out, pos, None, None, back)
    want = out[pos.long()].double().sum(1)
    assert bool(((back.double() - want).abs() <= 2.0 ** -8 * want.abs() + 4 * U * out[pos.long()].double().abs().sum(1) * 2).all())
    grad_w = torch.empty(16, 4, device="cuda")
    skg.skg_experts_combine_grad(back, out, pos, torch.full((16, 4), 2.0, device="cuda"), out, grad_w)
    assert torch.equal(out[M - 64:], (2 * back).repeat_interleave(4, 0))


@pytest.mark.parametrize("launch", [(1, 64, 1), (2, 128, 1), (2, 256, 1)])
def test_projection_to_more_than_31_bits_of_outputs(launch):
    M, N, K = 2 ** 18, 8200, 16
    g = torch.Generator().manual_seed(10)
    x = (torch.randn(M, K, generator=g) * 100).clamp(-448, 448).to(R.F8).cuda()
    W = (torch.randn(N, K, generator=g) * 100).clamp(-448, 448).to(R.F8).cuda()
    xs, ws = torch.rand(M, 1, generator=g).cuda(), torch.rand(R.blocks(N), 1, generator=g).cuda()
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    plan = skg.F8Plan(M, N, K, "bf16")
    plan.force(*launch)
    plan.run(x, xs, W, ws, None, y)
    plan.check()
    for s in (slice(0, 300), slice(M - 300, M)):
        R.check_linear(x[s], xs[s], W, ws, None, y[s])


def test_experts_whose_weights_are_more_than_32_bits():
    E, N, K, M = 300, 2048, 8192, 24
    W = torch.randint(0, 120, (E, N, K), dtype=torch.uint8, device="cuda").view(R.F8)
    g = torch.Generator().manual_seed(11)
    x = (torch.randn(M, K, generator=g) * 100).clamp(-448, 448).to(R.F8).cuda()
    xs, ws = torch.rand(M, 64, generator=g).cuda(), torch.rand(E, 16, 64, generator=g).cuda()
    counts = torch.zeros(E, dtype=torch.int32)
    counts[[0, 150, 298, 299]] = torch.tensor([2, 3, 1, 18], dtype=torch.int32)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int32), counts.cumsum(0).int()]).cuda()
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    plan = skg.F8Plan(M, N, K, "bf16", experts=E)
    plan.run(x, xs, W, ws, None, y, offsets=offsets)
    plan.check()
    at = offsets.tolist()
    for e in (0, 150, 298, 299):
        s = slice(at[e], at[e + 1])
        R.check_linear(x[s], xs[s], W[e], ws[e], None, y[s])


# --------------------------------------------------------------------------------- ends of the sizes
@pytest.mark.parametrize("launch", [None, (1, 16, 8), (1, 64, 1), (2, 128, 4), (2, 256, 1)])
def test_longest_k(launch):
    M, N, K = 3, 130, 131072
    g = torch.Generator().manual_seed(12)
    x = (torch.randn(M, K, generator=g) * 100).clamp(-448, 448).to(R.F8).cuda()
    W = (torch.randn(N, K, generator=g) * 100).clamp(-448, 448).to(R.F8).cuda()
    xs, ws = torch.rand(M, K // 128, generator=g).cuda(), torch.rand(2, K // 128, generator=g).cuda()
    y = torch.empty(M, N, device="cuda")
    plan = skg.F8Plan(M, N, K, "fp32")
    if launch:
        plan.force(*launch)
    plan.run(x, xs, W, ws, None, y)
    plan.check()
    R.check_linear(x, xs, W, ws, None, y)


@pytest.mark.parametrize("experts", [0, 1024])
def test_most_rows(experts):
    M, N, K = 2 ** 20, 40, 48
    g = torch.Generator().manual_seed(13)
    x = (torch.randn(M, K, generator=g) * 100).clamp(-448, 448).to(R.F8).cuda()
    W = (torch.randn(max(1, experts), N, K, generator=g) * 100).clamp(-448, 448).to(R.F8).cuda()
    xs, ws = torch.rand(M, 1, generator=g).cuda(), torch.rand(max(1, experts), 1, 1, generator=g).cuda()
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    plan = skg.F8Plan(M, N, K, "bf16", experts=experts)
    if not experts:
        plan.run(x, xs, W[0], ws[0], None, y)
        plan.check()
        R.check_linear(x, xs, W[0], ws[0], None, y)
        return
    cuts = torch.sort(torch.randint(0, M + 1, (experts - 1,), generator=g)).values.int()
    offsets = torch.cat([torch.zeros(1, dtype=torch.int32), cuts, torch.full((1,), M, dtype=torch.int32)]).cuda()
    plan.run(x, xs, W, ws, None, y, offsets=offsets)
    plan.check()
    at = offsets.tolist()
    for e in range(experts):
        s = slice(at[e], at[e + 1])
        if s.stop > s.start:
            R.check_linear(x[s], xs[s], W[e], ws[e], None, y[s])


def test_most_channels():
    """All weights but those of some channels are zeros."""
    N, K = 2 ** 31 - 256, 16
    at = torch.tensor([0, 127, 128, 2 ** 30 + 5, N - 257, N - 128, N - 1], device="cuda")
    g = torch.Generator().manual_seed(14)
    rows = (torch.randn(len(at), K, generator=g) * 100).clamp(-448, 448).to(R.F8).cuda()
    W = torch.zeros(N, K, dtype=torch.uint8, device="cuda")
    W[at] = rows.view(torch.uint8)
    x = (torch.randn(1, K, generator=g) * 100).clamp(-448, 448).to(R.F8).cuda()
    xs, ws = torch.ones(1, 1, device="cuda"), torch.ones(R.blocks(N), 1, device="cuda")
    y = torch.full((1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    plan = skg.F8Plan(1, N, K, "bf16")
    plan.run(x, xs, W.view(R.F8), ws, None, y)
    plan.check()
    R.check_linear(x, xs, rows, torch.ones(1, 1, device="cuda"), None, y[:, at])
    assert int((y != 0).sum()) == int((y[:, at] != 0).sum())


def test_longest_row_to_quantise():
    K = 2 ** 30
    x = torch.empty(1, K, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(15))
    q, s = torch.empty(1, K, dtype=R.F8, device="cuda"), torch.empty(1, K // 128, device="cuda")
    skg.skg_quantize_f8(x, None, q, s)
    for a in (0, K // 2, K - 2 ** 16):
        p = slice(a, a + 2 ** 16)
        R.check_quantised(x[:, p], q[:, p].contiguous(), s[:, a // 128:a // 128 + 512])


def test_sort_of_the_most_choices():
    T, k, E = 2 ** 21, 8, 1000
    expert = torch.randint(-1, E, (T, k), generator=torch.Generator(device="cuda").manual_seed(16), device="cuda", dtype=torch.int32)
    offsets = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    rows, pos = torch.empty(T * k, dtype=torch.int32, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda")
    skg.skg_experts_sort(expert, offsets, rows, pos)
    key = torch.where(expert.flatten() >= 0, expert.flatten(), E).long()
    order = torch.sort(key, stable=True).indices
    n = int((key < E).sum())
    assert torch.equal(offsets[1:].long(), torch.bincount(key, minlength=E + 1)[:E].cumsum(0)) and int(offsets[0]) == 0
    assert torch.equal(rows[:n].long(), order[:n] // k) and bool((rows[n:] == -1).all())
    want = torch.full((T * k,), -1, dtype=torch.long, device="cuda")
    want[order[:n]] = torch.arange(n, device="cuda")
    assert torch.equal(pos.flatten().long(), want)
