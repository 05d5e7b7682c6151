"""The example layer of experts on a stream that is not the current one."""
import pytest
import torch

from projection_gemm_gb300 import build, skg
from projection_gemm_gb300.f8_experts import F8Experts

pytestmark = pytest.mark.gpu

T, K_BEST, E, HIDDEN, INNER = 6, 2, 8, 256, 128
LONG = 40_000_000           # cycles of a stream that is busy: about 20 ms


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    skg.load()


def weights():
    g = torch.Generator().manual_seed(1)

    def normal(*shape):
        return (torch.randn(*shape, generator=g) * HIDDEN ** -0.5).to(torch.bfloat16).cuda()

    return normal(E, 2 * INNER, HIDDEN), normal(E, HIDDEN, INNER), normal(E, HIDDEN)


@pytest.mark.parametrize("handle", [False, True])
def test_route_reads_its_own_scores_on_the_given_stream(handle):
    """The choice of experts waits for the router's scores although its stream is behind the current one."""
    layer = F8Experts(T, K_BEST, *weights())
    x = torch.randn(T, HIDDEN, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    want_expert, want_weight = (t.clone() for t in layer.route(x))
    layer.scores.zero_()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(LONG)
    expert, weight = layer.route(x, stream=side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    assert torch.equal(expert, want_expert) and torch.equal(weight, want_weight)
    layer.check()
    layer.close()


def test_a_new_layer_is_there_for_a_step_on_any_stream(monkeypatch):
    """What it starts its buffers with has been written when it is handed out, so that it cannot land in a step's."""
    given = weights()
    zeros = torch.zeros

    def late(*args, **kw):
        torch.cuda._sleep(LONG)
        return zeros(*args, **kw)

    monkeypatch.setattr(torch, "zeros", late)
    layer = F8Experts(T, K_BEST, *given)
    assert torch.cuda.current_stream().query()
    layer.close()
