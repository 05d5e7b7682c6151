"""Python binding of libskg.so (see include/skg.h) -- argument marshalling only.

Every function here has the name of the C entry point it calls and does
nothing but convert arguments: torch tensors become device pointers, streams
become cudaStream_t handles, statuses become exceptions.  All computation
happens in the library's CUDA kernels; if the library is missing this module
raises instead of computing anything another way.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "lib", "libskg.so")

SKG_OK = 0
SKG_ERR_INVALID_ARG = 1
SKG_ERR_UNSUPPORTED = 2
SKG_ERR_ALIGNMENT = 3
SKG_ERR_CUDA = 4
SKG_ERR_DEVICE_TIMEOUT = 5

SKG_EPI_BF16 = 0
SKG_EPI_BF16_RESIDUAL = 1
SKG_EPI_FP32 = 2
EPILOGUES = {"bf16": SKG_EPI_BF16, "bf16_residual": SKG_EPI_BF16_RESIDUAL, "fp32": SKG_EPI_FP32}

CANONICAL_CHUNKS = 16     # SKG_CANONICAL_CHUNKS of include/skg.h

SKG_KERNEL_GEMV = 1
SKG_KERNEL_SPLITK_TC = 2
KERNEL_NAMES = {SKG_KERNEL_GEMV: "gemv", SKG_KERNEL_SPLITK_TC: "splitk_tc"}

SKG_Q8_KERNEL_STREAM = 1
SKG_Q8_KERNEL_SPLIT = 2
SKG_Q8_KERNEL_WIDE = 3
Q8_KERNEL_NAMES = {SKG_Q8_KERNEL_STREAM: "q8_stream", SKG_Q8_KERNEL_SPLIT: "q8_split",
                   SKG_Q8_KERNEL_WIDE: "q8_wide"}

# Every symbol include/skg.h declares.
EXPORTS = (
    "skg_plan_query", "skg_plan", "skg_plan_force", "skg_plan_force_kernel", "skg_plan_set_pdl", "skg_run",
    "skg_prefetch_l2", "skg_plan_set_prefetch_fraction", "skg_plan_info", "skg_plan_check",
    "skg_plan_destroy", "skg_debug_wait_timeout", "skg_last_error", "skg_version",
    "skg_run_noalloc", "skg_noalloc_check", "skg_plan_set_k_shard", "skg_combine_partials", "skg_plan_set_l2_ahead", "skg_plan_set_next_weight",
    "skg_plan_set_reducers",
    "skg_group", "skg_group_run", "skg_group_info", "skg_group_check", "skg_group_destroy",
    "skg_rmsnorm_q8", "skg_quantize_q8", "skg_q8_plan_query", "skg_q8_plan", "skg_q8_run", "skg_q8_plan_destroy",
    "skg_q8_plan_force", "skg_q8_plan_info", "skg_q8_plan_check", "skg_q8_debug_wait_timeout",
)


class SkgError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"skg status {status}: {message}")
        self.status = status


class skg_plan_desc(ctypes.Structure):
    _fields_ = [
        ("kernel_kind", ctypes.c_int), ("M", ctypes.c_int), ("N", ctypes.c_int),
        ("K", ctypes.c_int), ("epilogue", ctypes.c_int), ("split_k", ctypes.c_int),
        ("tile_n", ctypes.c_int), ("m_pad", ctypes.c_int), ("stages", ctypes.c_int),
        ("tma_burst", ctypes.c_int),
        ("grid", ctypes.c_int), ("threads", ctypes.c_int), ("smem_bytes", ctypes.c_int),
        ("from_table", ctypes.c_int), ("workspace_bytes", ctypes.c_size_t),
        ("prefetch_bytes", ctypes.c_size_t), ("pdl", ctypes.c_int), ("l2_ahead", ctypes.c_int),
        ("reducers", ctypes.c_int), ("ctas_per_sm", ctypes.c_int),
    ]

    def as_dict(self) -> dict:
        d = {f: getattr(self, f) for f, _ in self._fields_}
        d["kernel"] = KERNEL_NAMES.get(self.kernel_kind, "?")
        return d


class skg_q8_plan_desc(ctypes.Structure):
    _fields_ = [
        *((f, ctypes.c_int) for f in (
            "kernel_kind", "M", "N", "K", "epilogue", "static_weights", "m_tile", "n_tile", "tiles", "split_k",
            "grid", "threads", "smem_bytes", "stages", "ctas_per_sm")),
        ("workspace_bytes", ctypes.c_size_t),
    ]

    def as_dict(self) -> dict:
        d = {f: getattr(self, f) for f, _ in self._fields_}
        d["kernel"] = Q8_KERNEL_NAMES.get(self.kernel_kind, "?")
        return d


_lib = None


def load(path: str = LIB_PATH):
    """Load libskg.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m projection_gemm_gb300.build` "
                           "(there is no other implementation of the projection)")
    lib = ctypes.CDLL(path)
    vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    P = ctypes.POINTER
    lib.skg_plan_query.argtypes = [i, i, i, i, i, sz, P(skg_plan_desc)]
    lib.skg_plan.argtypes = [i, i, i, i, P(vp)]
    lib.skg_plan_force.argtypes = [vp, i, i, i, i]
    lib.skg_plan_set_pdl.argtypes = [vp, i]
    lib.skg_plan_force_kernel.argtypes = [vp, i]
    lib.skg_run.argtypes = [vp, vp, vp, vp, vp, vp]
    lib.skg_prefetch_l2.argtypes = [vp, vp, vp]
    lib.skg_plan_set_prefetch_fraction.argtypes = [vp, ctypes.c_double]
    lib.skg_plan_info.argtypes = [vp, P(skg_plan_desc)]
    lib.skg_plan_check.argtypes = [vp]
    lib.skg_plan_destroy.argtypes = [vp]
    lib.skg_debug_wait_timeout.argtypes = [vp, ctypes.c_ulonglong, vp]
    lib.skg_run_noalloc.argtypes = [i, i, i, i, vp, vp, vp, vp, vp]
    lib.skg_noalloc_check.argtypes = [vp]
    lib.skg_plan_set_k_shard.argtypes = [vp, i, i]
    lib.skg_combine_partials.argtypes = [i, i, i, P(vp), vp, vp, i, vp]
    lib.skg_plan_set_l2_ahead.argtypes = [vp, i]
    lib.skg_plan_set_reducers.argtypes = [vp, i]
    lib.skg_plan_set_next_weight.argtypes = [vp, vp, sz]
    lib.skg_group.argtypes = [i, i, P(i), P(i), P(i), P(i), P(vp)]
    lib.skg_group_run.argtypes = [vp, P(vp), P(vp), P(vp), P(vp), vp]
    lib.skg_group_info.argtypes = [vp, P(i), P(i), P(i), P(i)]
    lib.skg_group_check.argtypes = [vp]
    lib.skg_group_destroy.argtypes = [vp]
    lib.skg_rmsnorm_q8.argtypes = [i, i, ctypes.c_float, vp, sz, vp, sz, vp, vp, sz, vp, vp, vp, vp]
    lib.skg_quantize_q8.argtypes = [i, i, vp, sz, vp, sz, vp, vp, vp]
    lib.skg_q8_plan_query.argtypes = [i, i, i, i, i, P(skg_q8_plan_desc)]
    lib.skg_q8_plan.argtypes = [i, i, i, i, i, P(vp)]
    lib.skg_q8_run.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp]
    lib.skg_q8_plan_destroy.argtypes = [vp]
    lib.skg_q8_plan_force.argtypes = [vp, i, i, i]
    lib.skg_q8_plan_info.argtypes = [vp, P(skg_q8_plan_desc)]
    lib.skg_q8_plan_check.argtypes = [vp]
    lib.skg_q8_debug_wait_timeout.argtypes = [vp, ctypes.c_ulonglong, vp]
    for name in EXPORTS:
        getattr(lib, name).restype = ctypes.c_int
    lib.skg_last_error.restype = ctypes.c_char_p
    lib.skg_last_error.argtypes = []
    lib.skg_version.argtypes = []
    _lib = lib
    return lib


def _check(status: int):
    if status != SKG_OK:
        raise SkgError(status, load().skg_last_error().decode(errors="replace"))


def _epi(epilogue) -> int:
    return EPILOGUES[epilogue] if isinstance(epilogue, str) else int(epilogue)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def skg_version() -> int:
    return int(load().skg_version())


def skg_last_error() -> str:
    return load().skg_last_error().decode(errors="replace")


def skg_plan_query(M: int, N: int, K: int, epilogue, num_sms: int, l2_bytes: int) -> dict:
    d = skg_plan_desc()
    _check(load().skg_plan_query(M, N, K, _epi(epilogue), num_sms, l2_bytes, ctypes.byref(d)))
    return d.as_dict()


def skg_plan(M: int, N: int, K: int, epilogue) -> int:
    h = ctypes.c_void_p()
    _check(load().skg_plan(M, N, K, _epi(epilogue), ctypes.byref(h)))
    return h.value


def skg_plan_force(plan: int, split_k: int = 0, stages: int = 0, grid: int = 0, tma_burst: int = 0):
    _check(load().skg_plan_force(plan, split_k, stages, grid, tma_burst))


def skg_plan_force_kernel(plan: int, kind: int):
    _check(load().skg_plan_force_kernel(plan, kind))


def skg_plan_set_pdl(plan: int, enable: bool):
    _check(load().skg_plan_set_pdl(plan, 1 if enable else 0))


def skg_plan_set_next_weight(plan: int, W_next, nbytes: int):
    _check(load().skg_plan_set_next_weight(plan, _ptr(W_next), int(nbytes)))


def skg_plan_set_l2_ahead(plan: int, ahead: int):
    _check(load().skg_plan_set_l2_ahead(plan, int(ahead)))


def skg_plan_set_reducers(plan: int, reducers: int):
    _check(load().skg_plan_set_reducers(plan, int(reducers)))


def skg_plan_set_prefetch_fraction(plan: int, fraction: float):
    _check(load().skg_plan_set_prefetch_fraction(plan, float(fraction)))


def skg_plan_set_k_shard(plan: int, rank: int, ranks: int):
    _check(load().skg_plan_set_k_shard(plan, int(rank), int(ranks)))


def skg_combine_partials(M: int, N: int, partials, residual, y, epilogue="bf16", stream=None):
    """partials: R fp32 [M, N] device tensors (or addresses), in rank order."""
    arr = (ctypes.c_void_p * len(partials))(*[_ptr(t) for t in partials])
    _check(load().skg_combine_partials(M, N, len(partials), arr, _ptr(residual), _ptr(y), _epi(epilogue),
                                       _stream(stream)))


def skg_plan_info(plan: int) -> dict:
    d = skg_plan_desc()
    _check(load().skg_plan_info(plan, ctypes.byref(d)))
    return d.as_dict()


def skg_run(plan: int, x, W, residual, y, stream=None):
    _check(load().skg_run(plan, _ptr(x), _ptr(W), _ptr(residual), _ptr(y), _stream(stream)))


def skg_prefetch_l2(plan_next: int, W_next, side_stream=None):
    _check(load().skg_prefetch_l2(plan_next, _ptr(W_next), _stream(side_stream)))


def skg_plan_check(plan: int):
    _check(load().skg_plan_check(plan))


def skg_plan_destroy(plan: int):
    _check(load().skg_plan_destroy(plan))


def skg_debug_wait_timeout(plan, timeout_ns: int, stream=None):
    """plan None: the timeout word of the allocation-free entry point."""
    _check(load().skg_debug_wait_timeout(plan, int(timeout_ns), _stream(stream)))


def skg_run_noalloc(M: int, N: int, K: int, epilogue, x, W, residual, y, stream=None):
    """The split-K projection without a plan and without allocating (fixed
    in-library scratch); see include/skg.h for its limits."""
    _check(load().skg_run_noalloc(M, N, K, _epi(epilogue), _ptr(x), _ptr(W), _ptr(residual), _ptr(y),
                                  _stream(stream)))


def skg_noalloc_check(stream=None):
    """Synchronise the stream; raise SKG_ERR_DEVICE_TIMEOUT if a kernel of
    skg_run_noalloc ran out of a bounded wait since the last check."""
    _check(load().skg_noalloc_check(_stream(stream)))


class Plan:
    """Owns one skg plan handle; methods forward to the C entry points."""

    def __init__(self, M: int, N: int, K: int, epilogue="bf16"):
        self.M, self.N, self.K = M, N, K
        self.epilogue = _epi(epilogue)
        self.handle = skg_plan(M, N, K, self.epilogue)

    def info(self) -> dict:
        return skg_plan_info(self.handle)

    def force(self, split_k: int = 0, stages: int = 0, grid: int = 0, tma_burst: int = 0):
        skg_plan_force(self.handle, split_k, stages, grid, tma_burst)

    def force_kernel(self, kind: int):
        skg_plan_force_kernel(self.handle, kind)

    def set_pdl(self, enable: bool):
        skg_plan_set_pdl(self.handle, enable)

    def set_next_weight(self, W_next, nbytes: int):
        skg_plan_set_next_weight(self.handle, W_next, nbytes)

    def set_l2_ahead(self, ahead: int):
        skg_plan_set_l2_ahead(self.handle, ahead)

    def set_reducers(self, reducers: int):
        skg_plan_set_reducers(self.handle, reducers)

    def set_k_shard(self, rank: int, ranks: int):
        skg_plan_set_k_shard(self.handle, rank, ranks)

    def run(self, x, W, residual, y, stream=None):
        skg_run(self.handle, x, W, residual, y, stream)

    def prefetch(self, W, side_stream=None):
        skg_prefetch_l2(self.handle, W, side_stream)

    def check(self):
        skg_plan_check(self.handle)

    def close(self):
        if self.handle:
            skg_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------------------------------------- groups
def _ints(vals):
    return (ctypes.c_int * len(vals))(*[int(v) for v in vals])


def _ptrs(vals):
    return (ctypes.c_void_p * len(vals))(*[_ptr(v) for v in vals])


def skg_group(M: int, N, K, epilogue, dep=None) -> int:
    g = ctypes.c_void_p()
    n = len(N)
    _check(load().skg_group(n, M, _ints(N), _ints(K), _ints([_epi(e) for e in epilogue]),
                            _ints(dep) if dep is not None else None, ctypes.byref(g)))
    return g.value


def skg_group_run(group: int, x, W, residual, y, stream=None):
    res = None if residual is None else _ptrs(residual)
    _check(load().skg_group_run(group, _ptrs(x), _ptrs(W), res, _ptrs(y), _stream(stream)))


def skg_group_info(group: int, n: int) -> dict:
    grid, stages, units = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    split = (ctypes.c_int * n)()
    _check(load().skg_group_info(group, ctypes.byref(grid), ctypes.byref(stages), ctypes.byref(units), split))
    return {"grid": grid.value, "stages": stages.value, "units": units.value, "split": list(split)}


def skg_group_check(group: int):
    _check(load().skg_group_check(group))


def skg_group_destroy(group: int):
    _check(load().skg_group_destroy(group))


class Group:
    """Several projections of one M in one persistent launch (skg_group)."""

    def __init__(self, M: int, N, K, epilogue, dep=None):
        self.n = len(N)
        self.handle = skg_group(M, N, K, epilogue, dep)

    def run(self, x, W, residual, y, stream=None):
        skg_group_run(self.handle, x, W, residual, y, stream)

    def info(self) -> dict:
        return skg_group_info(self.handle, self.n)

    def check(self):
        skg_group_check(self.handle)

    def close(self):
        if self.handle:
            skg_group_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------------------------------ the 8-bit path
def _bad(what: str):
    raise SkgError(SKG_ERR_INVALID_ARG, what)


def _int(v, name) -> int:
    """A size or selector for the C ABI, whose int ctypes would otherwise cut to 32 bits."""
    if not -2**31 <= v < 2**31:
        _bad(f"{name} = {v} does not fit 32 bits")
    return v


def _rows(t, name, shape, dtype) -> int:
    """Row stride of a tensor of `shape` [M, K] whose rows are contiguous."""
    if t.dtype is not dtype or t.shape != shape or not t.is_cuda:
        _bad(f"{name} must be a CUDA tensor {list(shape)} of {dtype}")
    if t.is_contiguous():
        return shape[1]
    ld, one = t.stride()
    if (one != 1 and shape[1] > 1) or ld < shape[1]:
        _bad(f"{name}: elements of a row must be contiguous and rows must not overlap")
    return ld


def _dense(t, name, shape, dtype) -> int:
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or not t.is_cuda:
        _bad(f"{name} must be a contiguous CUDA tensor {list(shape)} of {dtype}")
    return t.data_ptr()


def _stream_of(stream, t):
    """The given stream, or the current one of t's device (the raw handle: a
    decode step's calls are short enough for a Stream object to show)."""
    if stream is not None:
        return _stream(stream)
    import torch
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def skg_rmsnorm_q8(x, residual, gamma, eps: float, h, q, scale, y=None, stream=None):
    """x, residual, h: bf16 [M, K] (rows may be strided); gamma bf16 [K]; q int8 [M, K];
    scale fp32 [M]; y bf16 [M, K].  residual, gamma, h and y may be None."""
    import torch
    bf16, shape = torch.bfloat16, x.shape
    if len(shape) != 2:
        _bad("x must be [M, K]")
    M, K = _int(shape[0], "M"), _int(shape[1], "K")
    ldx = _rows(x, "x", shape, bf16)
    ldr = 0 if residual is None else _rows(residual, "residual", shape, bf16)
    ldh = 0 if h is None else _rows(h, "h", shape, bf16)
    _check(load().skg_rmsnorm_q8(
        M, K, eps, x.data_ptr(), ldx, None if residual is None else residual.data_ptr(), ldr,
        None if gamma is None else _dense(gamma, "gamma", (K,), bf16), None if h is None else h.data_ptr(), ldh,
        None if y is None else _dense(y, "y", shape, bf16), _dense(q, "q", shape, torch.int8),
        _dense(scale, "scale", (M,), torch.float32), _stream_of(stream, x)))


def skg_quantize_q8(x, gate, q, scale, stream=None):
    """x, gate: bf16 [M, K] (rows may be strided; gate may be None); q int8 [M, K]; scale fp32 [M]."""
    import torch
    shape = x.shape
    if len(shape) != 2:
        _bad("x must be [M, K]")
    M, K = _int(shape[0], "M"), _int(shape[1], "K")
    ldx = _rows(x, "x", shape, torch.bfloat16)
    ldg = 0 if gate is None else _rows(gate, "gate", shape, torch.bfloat16)
    _check(load().skg_quantize_q8(
        M, K, x.data_ptr(), ldx, None if gate is None else gate.data_ptr(), ldg, _dense(q, "q", shape, torch.int8),
        _dense(scale, "scale", (M,), torch.float32), _stream_of(stream, x)))


def skg_q8_plan_query(M: int, N: int, K: int, epilogue, num_sms: int) -> dict:
    d = skg_q8_plan_desc()
    _check(load().skg_q8_plan_query(_int(M, "M"), _int(N, "N"), _int(K, "K"), _int(_epi(epilogue), "epilogue"),
                                    _int(num_sms, "num_sms"), ctypes.byref(d)))
    return d.as_dict()


def skg_q8_plan(M: int, N: int, K: int, epilogue, static_weights: bool = False) -> int:
    h = ctypes.c_void_p()
    _check(load().skg_q8_plan(_int(M, "M"), _int(N, "N"), _int(K, "K"), _int(_epi(epilogue), "epilogue"),
                              1 if static_weights else 0, ctypes.byref(h)))
    return h.value


def skg_q8_run(plan: int, x, x_scale, W, w_scale, residual, y, stream=None):
    _check(load().skg_q8_run(plan, _ptr(x), _ptr(x_scale), _ptr(W), _ptr(w_scale), _ptr(residual), _ptr(y),
                             _stream(stream)))


def skg_q8_plan_force(plan: int, kind: int = 0, m_tile: int = 0, split_k: int = 0):
    _check(load().skg_q8_plan_force(plan, _int(kind, "kind"), _int(m_tile, "m_tile"), _int(split_k, "split_k")))


def skg_q8_plan_info(plan: int) -> dict:
    d = skg_q8_plan_desc()
    _check(load().skg_q8_plan_info(plan, ctypes.byref(d)))
    return d.as_dict()


def skg_q8_plan_check(plan: int):
    _check(load().skg_q8_plan_check(plan))


def skg_q8_debug_wait_timeout(plan: int, timeout_ns: int, stream=None):
    _check(load().skg_q8_debug_wait_timeout(plan, int(timeout_ns), _stream(stream)))


def skg_q8_plan_destroy(plan: int):
    _check(load().skg_q8_plan_destroy(plan))


class Q8Plan:
    """Owns one 8-bit projection plan; run checks the tensors against it."""

    def __init__(self, M: int, N: int, K: int, epilogue="bf16", static_weights: bool = False):
        import torch
        self.M, self.N, self.K = M, N, K
        self.epilogue = _epi(epilogue)
        self._shapes = (M, K), (M,), (N, K), (N,), (M, N)
        self._types = (torch.int8, torch.float32, torch.bfloat16,
                       torch.float32 if self.epilogue == SKG_EPI_FP32 else torch.bfloat16)
        self.handle = None
        self.handle = skg_q8_plan(M, N, K, self.epilogue, static_weights)

    def run(self, x, x_scale, W, w_scale, residual, y, stream=None):
        # At few tokens the GPU takes a few microseconds a call, so the checks are
        # one expression (a call a tensor: 4.9 us a run instead of 4.6); what it
        # refuses is then named.
        mk, m, nk, n, mn = self._shapes
        i8, f32, bf16, out = self._types
        if not (x.dtype is i8 and x.shape == mk and x.is_contiguous() and x.is_cuda and
                W.dtype is i8 and W.shape == nk and W.is_contiguous() and W.is_cuda and
                x_scale.dtype is f32 and x_scale.shape == m and x_scale.is_contiguous() and x_scale.is_cuda and
                w_scale.dtype is f32 and w_scale.shape == n and w_scale.is_contiguous() and w_scale.is_cuda and
                y.dtype is out and y.shape == mn and y.is_contiguous() and y.is_cuda):
            for t, name, shape, dtype in ((x, "x", mk, i8), (x_scale, "x_scale", m, f32), (W, "W", nk, i8),
                                          (w_scale, "w_scale", n, f32), (y, "y", mn, out)):
                _dense(t, name, shape, dtype)
        if residual is not None:
            _dense(residual, "residual", mn, bf16)
        status = load().skg_q8_run(self.handle, x.data_ptr(), x_scale.data_ptr(), W.data_ptr(), w_scale.data_ptr(),
                                   None if residual is None else residual.data_ptr(), y.data_ptr(), _stream_of(stream, x))
        if status:
            _check(status)

    def force(self, kind: int = 0, m_tile: int = 0, split_k: int = 0):
        skg_q8_plan_force(self.handle, kind, m_tile, split_k)

    def info(self) -> dict:
        return skg_q8_plan_info(self.handle)

    def check(self):
        skg_q8_plan_check(self.handle)

    def close(self):
        if self.handle:
            skg_q8_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
