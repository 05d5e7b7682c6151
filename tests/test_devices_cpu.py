"""Tensors of another device than the current one, or than each other: refused by the
binding before the library is called.  Without a GPU: the tensors, the current
device and the library are stand-ins."""
import pytest
import torch

from projection_gemm_gb300 import skg

BF, F32, I32, F8, I8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn, torch.int8


class OnDevice:
    """What the binding asks of a tensor."""

    is_cuda = True

    def __init__(self, dtype, *shape):
        self.dtype, self.shape, self.device = dtype, torch.Size(shape), 0

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return True

    def stride(self):
        return self.shape[1], 1

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 1 << 20


class Library:
    """Counts the calls that reach it."""

    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*args):
            self.calls += 1
            return skg.SKG_OK
        return call


def f8_plan(epilogue, experts):
    plan = object.__new__(skg.F8Plan)
    each = (experts,) if experts else ()
    plan.experts, plan.handle = experts, None
    plan._shapes = (4, 256), (4, 2), (*each, 128, 256), (*each, 1, 2), (4, 128)
    plan._types = F8, F32, BF, I32, BF
    return plan


def q8_plan():
    plan = object.__new__(skg.Q8Plan)
    plan.handle = None
    plan._shapes = (4, 256), (4,), (128, 256), (128,), (4, 128)
    plan._types = I8, F32, BF, BF
    return plan


T = OnDevice
CALLS = {
    "rmsnorm_q8": (lambda x, r, g, h, q, s, y, stream=None: skg.skg_rmsnorm_q8(x, r, g, 1e-6, h, q, s, y, stream),
                   lambda: [T(BF, 4, 256), T(BF, 4, 256), T(BF, 256), T(BF, 4, 256), T(I8, 4, 256), T(F32, 4), T(BF, 4, 256)]),
    "quantize_q8": (skg.skg_quantize_q8, lambda: [T(BF, 4, 256), T(BF, 4, 256), T(I8, 4, 256), T(F32, 4)]),
    "Q8Plan.run": (q8_plan().run, lambda: [T(I8, 4, 256), T(F32, 4), T(I8, 128, 256), T(F32, 128), T(BF, 4, 128), T(BF, 4, 128)]),
    "quantize_f8": (skg.skg_quantize_f8, lambda: [T(BF, 4, 256), T(BF, 4, 256), T(F8, 6, 256), T(F32, 6, 2), T(I32, 6)]),
    "quantize_f8_weights": (skg.skg_quantize_f8_weights, lambda: [T(BF, 3, 200, 256), T(F8, 3, 200, 256), T(F32, 3, 2, 2)]),
    "F8Plan.run": (f8_plan("bf16_residual", 3).run, lambda: [T(F8, 4, 256), T(F32, 4, 2), T(F8, 3, 128, 256), T(F32, 3, 1, 2),
                                                             T(BF, 4, 128), T(BF, 4, 128), T(I32, 4)]),
    "experts_sort": (skg.skg_experts_sort, lambda: [T(I32, 4, 2), T(I32, 6), T(I32, 8), T(I32, 4, 2)]),
    "experts_gather": (skg.skg_experts_gather, lambda: [T(BF, 4, 64), T(I32, 8), T(BF, 8, 64)]),
    "experts_combine": (skg.skg_experts_combine, lambda: [T(BF, 8, 64), T(I32, 4, 2), T(F32, 4, 2), T(BF, 4, 64), T(BF, 4, 64)]),
    "experts_combine_grad": (skg.skg_experts_combine_grad, lambda: [T(BF, 4, 64), T(BF, 8, 64), T(I32, 4, 2), T(F32, 4, 2),
                                                                    T(BF, 8, 64), T(F32, 4, 2)]),
}
EACH = [(name, i) for name, (_, tensors) in CALLS.items() for i in range(len(tensors()))]


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(skg, "load", lambda: lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    return lib


@pytest.mark.parametrize("stream", [None, 0, 77])
@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_the_current_device_are_taken(name, stream, library):
    call, tensors = CALLS[name]
    call(*tensors(), stream=stream)
    assert library.calls == 1


@pytest.mark.parametrize("stream", [None, 0, 77])
@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_another_device_than_the_current_one_are_refused(name, stream, library):
    call, tensors = CALLS[name]
    given = tensors()
    for t in given:
        t.device = 1
    with pytest.raises(skg.SkgError) as e:
        call(*given, stream=stream)
    assert e.value.status == skg.SKG_ERR_INVALID_ARG and "device" in str(e.value) and library.calls == 0


@pytest.mark.parametrize("name,i", EACH)
def test_a_tensor_of_another_device_than_the_others_is_refused(name, i, library):
    call, tensors = CALLS[name]
    given = tensors()
    given[i].device = 1
    with pytest.raises(skg.SkgError) as e:
        call(*given)
    assert e.value.status == skg.SKG_ERR_INVALID_ARG and "device" in str(e.value) and library.calls == 0
