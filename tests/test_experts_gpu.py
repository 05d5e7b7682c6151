"""Tokens to their experts and back on a GB300: the sort against a stable sort, the
rows moved bit for bit, combinations and gradients against 64 bits.

A combination adds k products and a residual in fp32 (u = 2^-24), one fused
multiplication and addition each, and is rounded once to bf16 (2^-8 of the value):
  |out - exact| <= (k + 1) u (|residual| + sum |w y|) (1 + 2^-8) + 2^-8 |exact|.
grad_y is one product and one rounding.  grad_weight sums N exact products (bf16) in
fp32, at most N / 256 + 8 in a row and 13 more to join the threads:
  |off| <= (N / 256 + 21) u sum |grad y|.
"""
import pytest
import torch

from projection_gemm_gb300 import skg

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from projection_gemm_gb300 import build
    build.build()
    skg.load()
    assert torch.cuda.is_available()


def gen(*key):
    return torch.Generator().manual_seed(hash(key) % 2 ** 31)


def normal(g, *shape):
    return torch.randn(*shape, generator=g).to(torch.bfloat16).cuda()


def sort(expert, E):
    T, k = expert.shape
    offsets = torch.full((E + 1,), -9, dtype=torch.int32, device="cuda")
    rows = torch.full((T * k,), -9, dtype=torch.int32, device="cuda")
    pos = torch.full((T, k), -9, dtype=torch.int32, device="cuda")
    skg.skg_experts_sort(expert.cuda(), offsets, rows, pos)
    return offsets, rows, pos


def check_sort(expert, E):
    T, k = expert.shape
    offsets, rows, pos = (t.cpu() for t in sort(expert, E))
    flat = expert.flatten().long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    assert torch.equal(offsets.long(), torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]))
    n = int(offsets[-1])
    want_pos = torch.full((T * k,), -1, dtype=torch.long)
    want_pos[order[:n]] = torch.arange(n)
    assert torch.equal(pos.flatten().long(), want_pos)
    assert torch.equal(rows[:n].long(), order[:n] // k) and bool((rows[n:] == -1).all())


@pytest.mark.parametrize("E", [1, 7, 64, 384, 1024])
@pytest.mark.parametrize("T,k", [(1, 1), (1, 8), (3, 5), (33, 4), (500, 8), (513, 8), (4097, 3), (8192, 8), (70001, 2)])
def test_sort(T, k, E):
    g = gen(1, T, k, E)
    check_sort(torch.randint(0, E, (T, k), generator=g, dtype=torch.int32), E)


@pytest.mark.parametrize("T,k,E", [(40, 4, 6), (3000, 6, 50)])
def test_sort_leaves_out_what_is_no_expert(T, k, E):
    g = gen(2, T)
    e = torch.randint(-2, E + 2, (T, k), generator=g, dtype=torch.int32)
    e[0, 0], e[1, 0] = -2 ** 31, 2 ** 31 - 1
    check_sort(e, E)
    check_sort(torch.full((T, k), -1, dtype=torch.int32), E)
    check_sort(torch.full((T, k), E - 1, dtype=torch.int32), E)


def test_sort_of_no_tokens():
    offsets, _, _ = sort(torch.empty(0, 4, dtype=torch.int32), 9)
    assert bool((offsets == 0).all())


SIZES = [1, 2, 4, 7, 8, 256, 1000, 1001, 1002, 1004, 4104]


@pytest.mark.parametrize("N", SIZES)
@pytest.mark.parametrize("T,R", [(1, 1), (5, 40), (300, 77)])
def test_gather(T, R, N):
    g = gen(3, T, R, N)
    x = normal(g, T, N)
    rows = torch.randint(-1, T + 1, (R,), generator=g, dtype=torch.int32)
    out = torch.full((R, N), 5.0, dtype=torch.bfloat16, device="cuda")
    skg.skg_experts_gather(x, rows.cuda(), out)
    live = ((rows >= 0) & (rows < T)).cuda()
    want = torch.where(live[:, None], x[rows.clamp(0, T - 1).long().cuda()], 0)
    assert torch.equal(out, want)


@pytest.mark.parametrize("N,ld,off", [(64, 72, 0), (64, 65, 1), (64, 66, 2), (64, 68, 4), (100, 300, 3), (256, 264, 8), (256, 264, 4)])
def test_strided_rows(N, ld, off):
    g = gen(4, N, ld)
    T, k = 12, 3
    y = normal(g, T * k * ld + off + N)[off:off + T * k * ld].as_strided((T * k, N), (ld, 1))
    rows = torch.randperm(T * k, generator=g).int().cuda()
    out = torch.empty(T * k, N, dtype=torch.bfloat16, device="cuda")
    skg.skg_experts_gather(y, rows, out)
    assert torch.equal(out, y[rows.long()])
    check_combine(y, rows.view(T, k), torch.rand(T, k, generator=g).cuda(), normal(g, T, N))
    check_grad(normal(g, T, N), y, rows.view(T, k), torch.rand(T, k, generator=g).cuda())


def picked(y, pos):
    R = y.shape[0]
    live = (pos >= 0) & (pos < R)
    return torch.where(live[..., None], y[pos.clamp(0, R - 1).long()].double(), 0.0), live


def check_combine(y, pos, weight, residual):
    T, k = pos.shape
    out = torch.full((T, y.shape[1]), 5.0, dtype=torch.bfloat16, device="cuda")
    skg.skg_experts_combine(y, pos, weight, residual, out)
    v, live = picked(y, pos)
    w = torch.ones(T, k, dtype=torch.float64, device="cuda") if weight is None else weight.double()
    w = torch.where(live, w, 0.0)[..., None]
    want, mass = (v * w).sum(1), (v * w).abs().sum(1)
    if residual is not None:
        want, mass = want + residual.double(), mass + residual.double().abs()
    tol = (k + 1) * U * mass * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
    assert bool(((out.double() - want).abs() <= tol).all())
    return out


@pytest.mark.parametrize("N", SIZES)
@pytest.mark.parametrize("T,k", [(1, 1), (1, 8), (5, 3), (130, 8), (20, 19)])
@pytest.mark.parametrize("weights,residual", [(True, True), (True, False), (False, False)])
def test_combine(T, k, N, weights, residual):
    g = gen(5, T, k, N)
    y = normal(g, T * k, N)
    pos = torch.randperm(T * k, generator=g).int().view(T, k)
    pos[torch.rand(T, k, generator=g) < 0.2] = -1
    check_combine(y, pos.cuda(), torch.randn(T, k, generator=g).cuda() if weights else None,
                  normal(g, T, N) if residual else None)


def test_combine_of_left_out_choices():
    """Neither their weights nor any row is read into the sum; a token without any has its residual, or zeros."""
    g = gen(6)
    T, k, N = 6, 4, 264
    y = normal(g, T * k, N)
    y[0] = float("nan")                       # nobody's
    pos = torch.arange(1, T * k + 1, dtype=torch.int32).view(T, k)
    pos[1] = -1
    pos[2, 1], pos[3, 0], pos[4, 2] = -2 ** 31, 2 ** 31 - 1, T * k
    pos[5, 3] = T * k
    weight = torch.rand(T, k, generator=g)
    weight[(pos < 0) | (pos >= T * k)] = float("nan")
    res = normal(g, T, N)
    out = check_combine(y, pos.cuda(), weight.cuda(), res)
    assert torch.equal(out[1], res[1])
    assert bool((check_combine(y, pos.cuda(), weight.cuda(), None)[1] == 0).all())
    inplace = res.clone()
    skg.skg_experts_combine(y, pos.cuda(), weight.cuda(), inplace, inplace)
    assert torch.equal(inplace, out)


def check_grad(grad_out, y, pos, weight):
    (T, k), (rows, N) = pos.shape, y.shape
    grad_y = torch.full((rows, N), 5.0, dtype=torch.bfloat16, device="cuda")
    grad_weight = torch.full((T, k), 5.0, device="cuda")
    skg.skg_experts_combine_grad(grad_out, y, pos, weight, grad_y, grad_weight)
    v, live = picked(y, pos)
    gd = grad_out.double()[:, None]
    tol = (N / 256 + 21) * U * (v * gd).abs().sum(2)
    assert bool(((grad_weight.double() - (v * gd).sum(2)).abs() <= tol).all())
    assert bool((grad_weight[~live] == 0).all())
    want = torch.full((rows, N), 5.0, dtype=torch.float64, device="cuda")
    want[pos[live].long()] = (weight.double()[..., None] * gd)[live]
    assert bool(((grad_y.double() - want).abs() <= (2.0 ** -8 + 2 * U) * want.abs()).all())
    return grad_y, grad_weight


@pytest.mark.parametrize("N", SIZES + [7168])
@pytest.mark.parametrize("T,k", [(1, 1), (1, 8), (5, 3), (130, 8), (20, 19)])
def test_combine_grad(T, k, N):
    g = gen(7, T, k, N)
    pos = torch.randperm(T * k, generator=g).int().view(T, k)
    pos[torch.rand(T, k, generator=g) < 0.2] = -1
    check_grad(normal(g, T, N), normal(g, T * k, N), pos.cuda(), torch.randn(T, k, generator=g).cuda())


def test_gradients_against_differences():
    """Of L = sum(c * combine(f(gather(x)), w)), f a multiple of each row: with bf16 powers of two every step is exact,
    so a difference of L is its derivative."""
    g = gen(8)
    T, k, E, N = 6, 3, 5, 16
    expert = torch.randint(-1, E, (T, k), generator=g, dtype=torch.int32)
    offsets, rows, pos = sort(expert, E)

    def powers(*shape):
        return (2.0 ** torch.randint(-2, 3, shape, generator=g)) * (1 - 2 * torch.randint(0, 2, shape, generator=g))

    x, c = powers(T, N).bfloat16().cuda(), powers(T, N).bfloat16().cuda()
    w, f = powers(T, k).float().cuda(), powers(T * k, 1).bfloat16().cuda()

    def loss(x, w):
        xs, out = torch.empty(T * k, N, dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)
        skg.skg_experts_gather(x, rows, xs)
        y = xs * f
        skg.skg_experts_combine(y, pos, w, None, out)
        return (out.double() * c.double()).sum().item(), y

    _, y = loss(x, w)
    grad_y = torch.zeros_like(y)
    grad_w = torch.empty_like(w)
    skg.skg_experts_combine_grad(c, y, pos, w, grad_y, grad_w)
    grad_x = torch.empty_like(x)
    skg.skg_experts_combine(grad_y * f, pos, None, None, grad_x)
    for t in range(T):
        for j in range(k):
            wp = w.clone()
            wp[t, j] *= 2
            diff = (loss(x, wp)[0] - loss(x, w)[0]) / w[t, j].item()
            # loss sums rounded outputs: T N of them, each off by 2^-8 of at most k * 4^4
            assert abs(diff - grad_w[t, j].item()) <= 2 * N * 2.0 ** -8 * k * 256 * 4 / abs(w[t, j].item())
        n = t % N
        xp = x.clone()
        xp[t, n] *= 2
        diff = (loss(xp, w)[0] - loss(x, w)[0]) / x[t, n].item()
        assert abs(diff - grad_x[t, n].item()) <= 2.0 ** -8 * (2 * k * 256 * 4 / abs(x[t, n].item()) + abs(diff))


def test_the_same_call_gives_the_same_bits():
    g = gen(9)
    T, k, N = 700, 8, 1031
    pos = torch.randperm(T * k, generator=g).int().view(T, k).cuda()
    y, go, w = normal(g, T * k, N), normal(g, T, N), torch.rand(T, k, generator=g).cuda()
    first = check_combine(y, pos, w, None), *check_grad(go, y, pos, w)
    for _ in range(3):
        again = check_combine(y, pos, w, None), *check_grad(go, y, pos, w)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("N", [1, 2, 4, 8, 1031, 2050, 5000, 7168])
@pytest.mark.parametrize("k", [1, 8, 19])
def test_combine_grad_in_place_of_y(N, k):
    g = gen(10, N, k)
    T = 37
    pos = torch.randperm(T * k, generator=g).int().view(T, k)
    pos[torch.rand(T, k, generator=g) < 0.2] = -1
    pos = pos.cuda()
    y, go, w = normal(g, T * k, N), normal(g, T, N), torch.randn(T, k, generator=g).cuda()
    want_y, want_w = check_grad(go, y, pos, w)
    nobody = torch.ones(T * k, dtype=torch.bool, device="cuda")
    nobody[pos[pos >= 0].long()] = False
    want_y[nobody] = y[nobody]
    both, grad_weight = y.clone(), torch.empty_like(w)
    skg.skg_experts_combine_grad(go, both, pos, w, both, grad_weight)
    assert torch.equal(both, want_y) and torch.equal(grad_weight, want_w)


@pytest.mark.parametrize("N", [1, 6, 1031, 7168])
def test_a_row_of_several_choices(N):
    """Combined as often as it is chosen; each element of its gradient is of one of those choices."""
    g = gen(11, N)
    T, k, rows = 50, 11, 9
    pos = torch.randint(0, rows, (T, k), generator=g, dtype=torch.int32).cuda()
    y, go, w = normal(g, rows, N), normal(g, T, N), torch.randn(T, k, generator=g).cuda()
    check_combine(y, pos, w, None)
    grad_y, grad_weight = torch.empty_like(y), torch.empty_like(w)
    skg.skg_experts_combine_grad(go, y, pos, w, grad_y, grad_weight)
    v, _ = picked(y, pos)
    gd = go.double()[:, None]
    tol = (N / 256 + 21) * U * (v * gd).abs().sum(2)
    assert bool(((grad_weight.double() - (v * gd).sum(2)).abs() <= tol).all())
    each = (w[..., None] * go[:, None]).bfloat16()          # one product, rounded once more: the kernel's two operations
    for r in range(rows):
        assert bool((each[pos == r] == grad_y[r]).any(0).all())
