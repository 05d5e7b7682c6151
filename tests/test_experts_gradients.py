"""Gradients of gather and combination against differences, exactly.

L = sum(c combine(f gather(x), w)) with x, f, w and c of +-1 and +-2 and three choices a
token: |w f x| <= 8, or 16 where one factor is doubled, so each sum of three is a whole
number of at most 32, each gradient one of at most 256, and all of it fits bf16 or
fp32 without a rounding.  L is linear in each weight and each element of x, so the
difference that doubling one makes, over its value, is the derivative: equal, not near.

The same check is made without a GPU of plain operators, right ones and wrong ones."""
import pytest
import torch

from projection_gemm_gb300 import build, skg

T, K, E, N = 6, 3, 5, 16


class Kernels:
    device = "cuda"

    def __init__(self):
        build.build()
        skg.load()

    def sort(self, expert):
        offsets = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        rows, pos = torch.empty(T * K, dtype=torch.int32, device="cuda"), torch.empty(T, K, dtype=torch.int32, device="cuda")
        skg.skg_experts_sort(expert, offsets, rows, pos)
        return rows, pos

    def gather(self, x, rows):
        out = torch.empty(len(rows), x.shape[1], dtype=x.dtype, device="cuda")
        skg.skg_experts_gather(x, rows, out)
        return out

    def combine(self, y, pos, w):
        out = torch.empty(len(pos), y.shape[1], dtype=y.dtype, device="cuda")
        skg.skg_experts_combine(y, pos, w, None, out)
        return out

    def combine_grad(self, grad, y, pos, w):
        grad_y, grad_w = torch.zeros_like(y), torch.empty_like(w)
        skg.skg_experts_combine_grad(grad, y, pos, w, grad_y, grad_w)
        return grad_y, grad_w


class Plain:
    device = "cpu"

    def sort(self, expert):
        at = [i for e in range(E) for i, v in enumerate(expert.flatten().tolist()) if v == e]
        rows = torch.tensor([i // K for i in at] + [-1] * (T * K - len(at)))
        pos = torch.full((T * K,), -1)
        pos[torch.tensor(at)] = torch.arange(len(at))
        return rows, pos.view(T, K)

    def gather(self, x, rows):
        return torch.where(rows[:, None] >= 0, x[rows.clamp(min=0)], 0)

    def combine(self, y, pos, w):
        v = torch.where(pos[..., None] >= 0, y[pos.clamp(min=0)].float(), 0.0)
        return (v if w is None else v * w[..., None]).sum(1).bfloat16()

    def combine_grad(self, grad, y, pos, w):
        grad_y, grad_w = torch.zeros_like(y), torch.zeros_like(w)
        for t, j in (pos >= 0).nonzero().tolist():
            grad_y[pos[t, j]] = (w[t, j] * grad[t].float()).bfloat16()
            grad_w[t, j] = (grad[t].float() * y[pos[t, j]].float()).sum()
        return grad_y, grad_w


def wrong(which, factor):
    """Plain operators with one gradient times `factor`."""
    ops = Plain()
    right = ops.combine_grad

    def combine_grad(*args):
        grad_y, grad_w = right(*args)
        return (grad_y * factor, grad_w) if which == "grad_y" else (grad_y, grad_w * factor)

    ops.combine_grad = combine_grad
    if which == "gather's":              # a combination without weights, of the gradients of the gathered rows
        ops.combine_grad = right
        combine = ops.combine
        ops.combine = lambda y, pos, w: combine(y, pos, w) * (factor if w is None else 1)
    return ops


def differ(ops, seed):
    """Gradients that are not what differences give: (of w, of x)."""
    g = torch.Generator().manual_seed(seed)

    def values(*shape, dtype=torch.bfloat16):
        return ((1 + torch.randint(0, 2, shape, generator=g)) * (1 - 2 * torch.randint(0, 2, shape, generator=g))).to(dtype).to(ops.device)

    expert = torch.randint(-1, E, (T, K), generator=g, dtype=torch.int32).to(ops.device)
    rows, pos = ops.sort(expert)
    x, c, f, w = values(T, N), values(T, N), values(T * K, 1), values(T, K, dtype=torch.float32)

    def loss(x, w):
        return (ops.combine(ops.gather(x, rows) * f, pos, w).double() * c.double()).sum().item()

    grad_y, grad_w = ops.combine_grad(c, ops.gather(x, rows) * f, pos, w)
    grad_x = ops.combine(grad_y * f, pos, None)
    base, bad_w, bad_x = loss(x, w), 0, 0
    for t in range(T):
        for j in range(K):
            more = w.clone()
            more[t, j] *= 2
            bad_w += (loss(x, more) - base) / w[t, j].item() != grad_w[t, j].item()
        for n in range(N):
            more = x.clone()
            more[t, n] *= 2
            bad_x += (loss(more, w) - base) / x[t, n].item() != grad_x[t, n].item()
    assert (expert >= 0).any() and (expert < 0).any()
    return bad_w, bad_x


@pytest.mark.parametrize("seed", range(4))
def test_plain_gradients_are_differences(seed):
    assert differ(Plain(), seed) == (0, 0)


@pytest.mark.parametrize("factor", [0, -1, 2])
@pytest.mark.parametrize("which", ["grad_y", "grad_weight", "gather's"])
def test_wrong_gradients_are_not(which, factor):
    bad_w, bad_x = differ(wrong(which, factor), 0)
    assert bad_w > 9 if which == "grad_weight" else bad_x > 60


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(4))
def test_gradients_are_differences(seed):
    assert differ(Kernels(), seed) == (0, 0)
