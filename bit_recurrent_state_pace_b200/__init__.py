"""Python binding of libpace (PACE periodic low-bit recurrent-state decode).

Argument marshalling only: every step of the decode path runs in the CUDA
kernels of ``libpace.so``.  PyTorch supplies device memory and streams.
The functions keep the C names of ``include/pace.h``; ``PacePool`` is a
convenience owner of the three device regions a pool needs.

Importing this package loads ``libpace.so`` from this directory and raises
``ImportError`` if it is missing (build it with
``python -m bit_recurrent_state_pace_b200.build``); there is no fallback.
"""
from __future__ import annotations

import ctypes
import operator
import os
import warnings
from typing import Optional, Sequence, Tuple

import torch

__all__ = [
    "PaceError", "lib", "LIB_PATH",
    "PACE_SCALE_COL", "PACE_SCALE_ROW", "PACE_IO_BF16", "PACE_IO_F32",
    "PACE_OK", "PACE_ERR_INVALID_ARG", "PACE_ERR_UNSUPPORTED", "PACE_ERR_CUDA", "PACE_ERR_DEVICE_FLAGS",
    "PACE_FLAG_NONFINITE", "PACE_FLAG_SCALE_OVERFLOW", "PACE_FLAG_BUFFER_FULL", "PACE_FLAG_TIMEOUT",
    "PACE_FILL_COMMIT",
    "pace_pool_bytes", "pace_init_pool", "pace_destroy_pool", "pace_pool_layout",
    "pace_pool_load", "pace_pool_export", "pace_decode_step", "pace_commit_period",
    "pace_decode_step_range", "pace_commit_period_range", "pace_decay_rates",
    "pace_select_head_bits", "pace_prefill", "pace_prefill_range", "pace_host_staging_bytes",
    "pace_decode_host", "pace_set_commit_threshold", "pace_window_scratch_bytes", "pace_window_step",
    "pace_window_step_static", "PACE_WINDOW_STATIC_SCRATCH_BYTES", "pace_set_commit_engine",
    "PACE_COMMIT_MMA", "PACE_COMMIT_TCGEN05", "pace_debug_wait_fault",
    "pace_quantize", "pace_dequantize", "pace_pool_status", "pace_pool_clear_status",
    "pace_gdn_step_f32", "pace_gdn_step_bf16", "pace_status_string", "pace_version",
    "PACE_NORM_L2", "PACE_NORM_RMS", "pace_linattn_workspace_bytes", "pace_linattn_forward",
    "pace_linattn_backward", "pace_linattn_step", "pace_debug_linattn_wait", "pace_qk_norm_workspace_bytes", "pace_qk_norm_rotate",
    "pace_qk_norm_rotate_backward",
    "PacePool",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libpace.so")

PACE_SCALE_COL, PACE_SCALE_ROW = 0, 1
PACE_IO_BF16, PACE_IO_F32 = 0, 1
PACE_FLAG_NONFINITE = 0x1
PACE_FLAG_SCALE_OVERFLOW = 0x2
PACE_FLAG_BUFFER_FULL = 0x4
PACE_FLAG_TIMEOUT = 0x8
PACE_FILL_COMMIT = 0x100
PACE_WINDOW_STATIC_SCRATCH_BYTES = 8 << 20
PACE_COMMIT_MMA, PACE_COMMIT_TCGEN05 = 0, 1
PACE_NORM_L2, PACE_NORM_RMS = 0, 1
PACE_OK, PACE_ERR_INVALID_ARG, PACE_ERR_UNSUPPORTED, PACE_ERR_CUDA, PACE_ERR_DEVICE_FLAGS = 0, 1, 2, 3, 4


class PaceError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {_status_name(status)} ({status})")
        self.status = status


class _Desc(ctypes.Structure):
    _fields_ = [("num_slots", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32), ("period", ctypes.c_int32),
                ("scale_axis", ctypes.c_int32), ("io_dtype", ctypes.c_int32),
                ("head_bits", ctypes.POINTER(ctypes.c_uint8)), ("buffer_e4m3", ctypes.c_int32)]


class _LinattnDesc(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32), ("io_dtype", ctypes.c_int32),
                ("total_tokens", ctypes.c_int64), ("max_len", ctypes.c_int64),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("o_stride", ctypes.c_int64)]


class _QkNormDesc(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int64), ("num_q_heads", ctypes.c_int32),
                ("num_k_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("norm", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("eps", ctypes.c_float), ("q_scale", ctypes.c_float),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("q_out_stride", ctypes.c_int64), ("k_out_stride", ctypes.c_int64)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libpace.so not found at {LIB_PATH}: build it with "
                          "`python -m bit_recurrent_state_pace_b200.build` (there is no CPU fallback)")
    L = ctypes.CDLL(LIB_PATH)
    P, S, I32, I64, U32p, U16p, F32p = (ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32,
                                        ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p)
    Sp = ctypes.POINTER(ctypes.c_size_t)
    sig = {
        "pace_pool_bytes": [ctypes.POINTER(_Desc), Sp, Sp, Sp],
        "pace_init_pool": [ctypes.POINTER(_Desc), P, P, P, P, ctypes.POINTER(ctypes.c_void_p)],
        "pace_pool_layout": [P, I32, Sp, Sp, Sp],
        "pace_pool_load": [P, F32p, P],
        "pace_pool_export": [P, F32p, P],
        "pace_decode_step": [P, P, P, P, P, P, F32p, P],
        "pace_commit_period": [P, P],
        "pace_decode_step_range": [P, I32, I32, I32, P, P, P, P, P, F32p, P],
        "pace_commit_period_range": [P, I32, I32, I32, P],
        "pace_decay_rates": [P, I64, I32, I32, P, P],
        "pace_prefill": [P, I64, P, P, P, P, P, F32p, P],
        "pace_host_staging_bytes": [P, Sp],
        "pace_set_commit_threshold": [P, ctypes.c_float],
        "pace_set_commit_engine": [P, I32],
        "pace_debug_wait_fault": [P, ctypes.c_uint64, ctypes.c_uint32],
        "pace_window_scratch_bytes": [P, Sp],
        "pace_window_step": [P, P, P, P, P, P, F32p, P, P],
        "pace_window_step_static": [P, P, P, P, P, P, F32p, P],
        "pace_decode_host": [P, I32, P, P, P, P, P, P, P, P, P, P],
        "pace_prefill_range": [P, I32, I32, I64, P, P, P, P, P, F32p, P],
        "pace_select_head_bits": [P, I32, I32, P],
        "pace_quantize": [F32p, I64, I32, I32, I32, I32, P, U16p, U32p, P],
        "pace_dequantize": [P, U16p, I64, I32, I32, I32, I32, F32p, P],
        "pace_pool_status": [P, P, ctypes.POINTER(ctypes.c_uint32)],
        "pace_pool_clear_status": [P, P],
        "pace_linattn_workspace_bytes": [ctypes.POINTER(_LinattnDesc), I32, Sp],
        "pace_linattn_forward": [ctypes.POINTER(_LinattnDesc)] + [P] * 11,
        "pace_linattn_backward": [ctypes.POINTER(_LinattnDesc)] + [P] * 15,
        "pace_linattn_step": [ctypes.POINTER(_LinattnDesc)] + [P] * 7,
        "pace_debug_linattn_wait": [ctypes.c_uint32, ctypes.c_uint32],
        "pace_qk_norm_workspace_bytes": [ctypes.POINTER(_QkNormDesc), Sp],
        "pace_qk_norm_rotate": [ctypes.POINTER(_QkNormDesc)] + [P] * 9,
        "pace_qk_norm_rotate_backward": [ctypes.POINTER(_QkNormDesc)] + [P] * 14,
        "pace_gdn_step_f32": [F32p, P, P, P, P, P, I32, F32p, I64, I32, I32, P],
        "pace_gdn_step_bf16": [U16p, P, P, P, P, P, I32, F32p, I64, I32, I32, P],
    }
    for name, args in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    L.pace_destroy_pool.argtypes = [P]
    L.pace_destroy_pool.restype = None
    L.pace_status_string.argtypes = [ctypes.c_int]
    L.pace_status_string.restype = ctypes.c_char_p
    L.pace_version.argtypes = []
    L.pace_version.restype = ctypes.c_char_p
    return L


lib = _load()


def _status_name(s: int) -> str:
    return lib.pace_status_string(int(s)).decode()


def _check(fn: str, status: int, ok=(PACE_OK,)) -> int:
    if status not in ok:
        raise PaceError(fn, status)
    return status


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libpace takes device tensors")
    if not t.is_contiguous():
        raise ValueError("libpace takes contiguous tensors")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _desc(B, H, d_k, d_v, P, axis, io, head_bits, buffer_e4m3=0) -> Tuple[_Desc, ctypes.Array]:
    vals = [int(b) for b in head_bits]
    bits_arr = (ctypes.c_uint8 * max(len(vals), 1))(*vals)
    d = _Desc(B, H, d_k, d_v, P, axis, io, ctypes.cast(bits_arr, ctypes.POINTER(ctypes.c_uint8)),
              int(buffer_e4m3))
    return d, bits_arr


# ---------------------------------------------------------------- C names

def pace_pool_bytes(B, H, d_k, d_v, P, axis, io, head_bits, buffer_e4m3=0) -> Tuple[int, int, int]:
    d, keep = _desc(B, H, d_k, d_v, P, axis, io, head_bits, buffer_e4m3)
    a, b, c = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check("pace_pool_bytes", lib.pace_pool_bytes(ctypes.byref(d), ctypes.byref(a), ctypes.byref(b),
                                                   ctypes.byref(c)))
    return a.value, b.value, c.value


def pace_init_pool(B, H, d_k, d_v, P, axis, io, head_bits, state, buffer, aux, stream=None,
                   buffer_e4m3=0) -> int:
    d, keep = _desc(B, H, d_k, d_v, P, axis, io, head_bits, buffer_e4m3)
    out = ctypes.c_void_p()
    _check("pace_init_pool", lib.pace_init_pool(ctypes.byref(d), _ptr(state), _ptr(buffer), _ptr(aux),
                                                 _stream(stream), ctypes.byref(out)))
    return out.value


def pace_destroy_pool(handle: int) -> None:
    lib.pace_destroy_pool(handle)


def pace_pool_layout(handle: int, head: int) -> Tuple[int, int, int]:
    a, b, c = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check("pace_pool_layout", lib.pace_pool_layout(handle, head, ctypes.byref(a), ctypes.byref(b),
                                                     ctypes.byref(c)))
    return a.value, b.value, c.value


def pace_pool_load(handle: int, S: torch.Tensor, stream=None) -> None:
    _check("pace_pool_load", lib.pace_pool_load(handle, _ptr(S), _stream(stream)))


def pace_pool_export(handle: int, S: torch.Tensor, stream=None) -> None:
    _check("pace_pool_export", lib.pace_pool_export(handle, _ptr(S), _stream(stream)))


def pace_decode_step(handle: int, q, k, v, alpha, beta, o, stream=None) -> None:
    _check("pace_decode_step", lib.pace_decode_step(handle, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                                                     _ptr(beta), _ptr(o), _stream(stream)))


def pace_commit_period(handle: int, stream=None) -> None:
    _check("pace_commit_period", lib.pace_commit_period(handle, _stream(stream)))


def pace_window_scratch_bytes(handle: int) -> int:
    n = ctypes.c_size_t()
    _check("pace_window_scratch_bytes", lib.pace_window_scratch_bytes(handle, ctypes.byref(n)))
    return n.value


def pace_window_step(handle: int, q, k, v, alpha, beta, o, scratch, stream=None) -> None:
    _check("pace_window_step", lib.pace_window_step(handle, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                                                    _ptr(beta), _ptr(o), _ptr(scratch), _stream(stream)))


def pace_window_step_static(handle: int, q, k, v, alpha, beta, o, stream=None) -> None:
    """pace_window_step with the library's own device scratch (no allocation)."""
    _check("pace_window_step_static", lib.pace_window_step_static(
        handle, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(o), _stream(stream)))


def pace_set_commit_threshold(handle: int, tau: float) -> None:
    _check("pace_set_commit_threshold", lib.pace_set_commit_threshold(handle, float(tau)))


def pace_set_commit_engine(handle: int, engine: int) -> None:
    _check("pace_set_commit_engine", lib.pace_set_commit_engine(handle, int(engine)))


def pace_debug_wait_fault(handle: int, wait_limit_ns: int, extra_tx_bytes: int) -> None:
    _check("pace_debug_wait_fault", lib.pace_debug_wait_fault(handle, int(wait_limit_ns), int(extra_tx_bytes)))


def pace_host_staging_bytes(handle: int) -> int:
    n = ctypes.c_size_t()
    _check("pace_host_staging_bytes", lib.pace_host_staging_bytes(handle, ctypes.byref(n)))
    return n.value


def _host_ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if t.is_cuda or not t.is_contiguous():
        raise ValueError("pace_decode_host takes contiguous host tensors")
    return t.data_ptr()


def pace_decode_host(handle: int, n_tokens: int, q, k, v, alpha, beta, o, staging, stream,
                     h2d_stream, d2h_stream) -> None:
    _check("pace_decode_host", lib.pace_decode_host(
        handle, n_tokens, _host_ptr(q), _host_ptr(k), _host_ptr(v), _host_ptr(alpha), _host_ptr(beta),
        _host_ptr(o), _ptr(staging), _stream(stream), _stream(h2d_stream), _stream(d2h_stream)))


def pace_prefill(handle: int, T: int, q, k, v, alpha, beta, o=None, stream=None) -> None:
    _check("pace_prefill", lib.pace_prefill(handle, T, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                                             _ptr(beta), _ptr(o), _stream(stream)))


def pace_prefill_range(handle: int, slot_begin: int, slot_count: int, T: int, q, k, v, alpha, beta,
                       o=None, stream=None) -> None:
    _check("pace_prefill_range", lib.pace_prefill_range(handle, slot_begin, slot_count, T, _ptr(q),
                                                         _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                                         _ptr(o), _stream(stream)))


def pace_decay_rates(alpha: torch.Tensor, num_heads: int, io: int, rates: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """Mean -ln(alpha) per head over the rows of a device gate matrix [rows][num_heads]."""
    if rates is None:
        rates = torch.empty(num_heads, dtype=torch.float64, device=alpha.device)
    rows = alpha.numel() // num_heads
    _check("pace_decay_rates", lib.pace_decay_rates(_ptr(alpha), rows, num_heads, io, _ptr(rates),
                                                     _stream(stream)))
    return rates


def pace_select_head_bits(rates: Sequence[float], num_int8: int) -> list:
    """Host: 8 bits for the num_int8 heads with the slowest decay, 4 for the rest."""
    vals = [float(r) for r in rates]
    arr = (ctypes.c_double * max(len(vals), 1))(*vals)
    out = (ctypes.c_uint8 * max(len(vals), 1))()
    _check("pace_select_head_bits", lib.pace_select_head_bits(
        ctypes.cast(arr, ctypes.c_void_p), len(vals), num_int8, ctypes.cast(out, ctypes.c_void_p)))
    return [int(out[i]) for i in range(len(vals))]


def pace_decode_step_range(handle: int, slot_begin: int, slot_count: int, blocks_per_sm: int,
                           q, k, v, alpha, beta, o, stream=None) -> None:
    _check("pace_decode_step_range",
           lib.pace_decode_step_range(handle, slot_begin, slot_count, blocks_per_sm, _ptr(q), _ptr(k),
                                      _ptr(v), _ptr(alpha), _ptr(beta), _ptr(o), _stream(stream)))


def pace_commit_period_range(handle: int, slot_begin: int, slot_count: int, blocks_per_sm: int,
                             stream=None) -> None:
    _check("pace_commit_period_range",
           lib.pace_commit_period_range(handle, slot_begin, slot_count, blocks_per_sm, _stream(stream)))


def pace_quantize(S, n_mats, d_k, d_v, bits, axis, codes, scales, flags=None, stream=None) -> None:
    _check("pace_quantize", lib.pace_quantize(_ptr(S), n_mats, d_k, d_v, bits, axis, _ptr(codes),
                                               _ptr(scales), _ptr(flags), _stream(stream)))


def pace_dequantize(codes, scales, n_mats, d_k, d_v, bits, axis, S, stream=None) -> None:
    _check("pace_dequantize", lib.pace_dequantize(_ptr(codes), _ptr(scales), n_mats, d_k, d_v, bits,
                                                   axis, _ptr(S), _stream(stream)))


def pace_pool_status(handle: int, stream=None) -> int:
    f = ctypes.c_uint32()
    _check("pace_pool_status", lib.pace_pool_status(handle, _stream(stream), ctypes.byref(f)),
           ok=(PACE_OK, PACE_ERR_DEVICE_FLAGS))
    return f.value


def pace_pool_clear_status(handle: int, stream=None) -> None:
    _check("pace_pool_clear_status", lib.pace_pool_clear_status(handle, _stream(stream)))


def pace_gdn_step_f32(S, q, k, v, alpha, beta, io, o, n, d_k, d_v, stream=None) -> None:
    _check("pace_gdn_step_f32", lib.pace_gdn_step_f32(_ptr(S), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                                                       _ptr(beta), io, _ptr(o), n, d_k, d_v,
                                                       _stream(stream)))


def pace_gdn_step_bf16(S, q, k, v, alpha, beta, io, o, n, d_k, d_v, stream=None) -> None:
    _check("pace_gdn_step_bf16", lib.pace_gdn_step_bf16(_ptr(S), _ptr(q), _ptr(k), _ptr(v),
                                                         _ptr(alpha), _ptr(beta), io, _ptr(o), n,
                                                         d_k, d_v, _stream(stream)))


# ------------------------------------------------ linear attention, query/key norms
#
# These calls check shapes, types and devices (the C entry points see pointers
# only), run on the device of their first tensor whichever device is current,
# allocate the outputs and the workspace that are not given, and return the
# outputs, which are detached: autograd records nothing (a warning says so where
# an input requires gradients; the _backward calls are for autograd functions).
# Token rows may lie apart (a part of a wider projection): the last
# two dimensions are dense, the row stride is free.

_IO_OF = {torch.bfloat16: PACE_IO_BF16, torch.float32: PACE_IO_F32}


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _rows(name: str, t: torch.Tensor, heads: int, d: int, like: torch.Tensor) -> Tuple[int, int]:
    """(rows, row stride in elements) of [..., heads, d] token rows."""
    _need(isinstance(t, torch.Tensor) and t.is_cuda and t.device == like.device, f"{name}: a tensor on {like.device}")
    _need(t.dtype == like.dtype, f"{name}: {like.dtype}, not {t.dtype}")
    sh, st = t.shape, t.stride()
    _need(len(sh) >= 3 and sh[-1] == d and sh[-2] == heads, f"{name}: [..., {heads}, {d}] rows, not {tuple(sh)}")
    rows = 1
    for x in sh[:-2]:
        rows *= x
    if rows * heads == 0:
        return rows, 0
    _need((d == 1 or st[-1] == 1) and (heads == 1 or st[-2] == d), f"{name}: each row's heads are contiguous")
    at = None                                   # the row stride; leading dimensions fold into one
    for x, s in zip(reversed(sh[:-2]), reversed(st[:-2])):
        if x == 1:
            continue
        if at is None:
            at, span = s, s * x
        else:
            _need(s == span, f"{name}: the leading dimensions lie at one stride")
            span = s * x
    _need(at is None or at >= heads * d, f"{name}: rows that do not overlap")
    return rows, 0 if at is None else at


def _plain(name: str, t: Optional[torch.Tensor], shape, dtype, like: torch.Tensor) -> Optional[int]:
    """Address of an optional contiguous tensor of that shape and type on the device of `like`."""
    if t is None:
        return None
    _need(isinstance(t, torch.Tensor) and t.is_cuda and t.device == like.device, f"{name}: a tensor on {like.device}")
    _need(t.dtype == dtype and tuple(t.shape) == tuple(shape) and t.is_contiguous(),
          f"{name}: contiguous {dtype} {tuple(shape)}, not {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # current_stream() without the wrapper object
_device_now = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)     # current_device() likewise


class _On:
    """Makes a device current for a call and gives the stream to launch on."""
    __slots__ = ("index", "stream", "back")

    def __init__(self, index: int, stream):
        self.index = index
        self.stream = stream

    def __enter__(self):
        self.back = torch.cuda.current_device()
        if self.back != self.index:
            torch.cuda.set_device(self.index)
        if self.stream is None and _raw_stream is not None:
            return _raw_stream(self.index)
        return _stream(self.stream)

    def __exit__(self, *exc):
        if self.back != self.index:
            torch.cuda.set_device(self.back)
        return False


def _run(name: str, fn, index: int, stream, *args) -> None:
    """fn(*args, stream) with device `index` current."""
    if stream is None and _raw_stream is not None and _device_now() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with _On(index, stream) as st:
            status = fn(*args, st)
    if status != PACE_OK:
        raise PaceError(name, status)


# What a call's shapes, strides, types and devices lead to (the checks passed, the descriptor, sizes), kept so that
# the next call of the same form pays for a lookup; no tensor and no address is kept.
_plans: dict = {}


def _whole(name: str, x) -> Optional[int]:
    """An optional integer as one: nothing else (a tensor, say) becomes part of a plan's key."""
    if x is None or type(x) is int:
        return x
    try:
        return operator.index(x)
    except TypeError:
        raise ValueError(f"{name}: an integer, not {type(x).__name__}") from None


def _number(name: str, x) -> float:
    """A real number as a float."""
    if type(x) is float:
        return x
    try:
        return float(x)
    except (TypeError, ValueError, RuntimeError):
        raise ValueError(f"{name}: a number, not {type(x).__name__}") from None


def _form(t):
    if t is None:
        return None
    try:
        return t.shape, t.stride(), t.dtype, t.get_device(), t.requires_grad
    except AttributeError:
        return type(t)                           # no tensor: the checks of a first call refuse it


def _plan(key, build):
    plan = _plans.get(key)
    if plan is None:
        plan = build()
        if len(_plans) >= 4096:
            _plans.clear()
        _plans[key] = plan
    return plan


def _wants_grad(*tensors) -> bool:
    """Of a plan's inputs: whether one requires gradients."""
    return any(t is not None and t.requires_grad for t in tensors)


def _detached(name: str) -> None:
    """Says so where autograd would be expected to record the call: the outputs are detached."""
    if torch.is_grad_enabled():
        warnings.warn(f"{name} records nothing for autograd, its outputs are detached from inputs that require gradients: "
                      f"call it in an autograd function (or under torch.no_grad())", stacklevel=3)


def _opt(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _new(shape, dtype, like: torch.Tensor, stream) -> torch.Tensor:
    """An output or workspace for work on `stream` (None: the current one) of the device of `like`."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), like.device)
    with torch.cuda.stream(s):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _like(t: torch.Tensor, stream) -> torch.Tensor:
    """A packed tensor of t's shape and type for work on `stream`."""
    if stream is None:
        return torch.empty_like(t, memory_format=torch.contiguous_format)
    return _new(t.shape, t.dtype, t, stream)


def _workspace(name: str, nbytes: int, given: Optional[torch.Tensor], like: torch.Tensor, stream):
    if given is None:
        return _new(nbytes, torch.uint8, like, stream) if nbytes else None
    _need(isinstance(given, torch.Tensor) and given.is_cuda and given.device == like.device and given.is_contiguous(),
          f"{name}: workspace: a contiguous tensor on {like.device}")
    _need(given.numel() * given.element_size() >= nbytes, f"{name}: workspace of {nbytes} bytes")
    return given


def _linattn(q, k, v, log_decay, num_seqs, max_len, cu_seqlens):
    """Descriptor and common checks; (desc, rows of q, N, H, d)."""
    _need(isinstance(q, torch.Tensor) and q.is_cuda, "libpace takes device tensors")
    _need(q.dtype in _IO_OF, f"q: bfloat16 or float32, not {q.dtype}")
    _need(q.dim() in (3, 4), "q: [tokens, heads, d] or [sequences, tokens, heads, d]")
    _need(log_decay is not None, "log_decay: the heads' log decays")
    H, d = q.shape[-2], q.shape[-1]
    total, qs = _rows("q", q, H, d, q)
    tk, ks = _rows("k", k, H, d, q)
    tv, vs = _rows("v", v, H, d, q)
    _need(tk == total and tv == total, "q, k and v: as many rows each")
    if cu_seqlens is not None:
        n = cu_seqlens.numel() - 1
        _need(num_seqs is None or num_seqs == n, "cu_seqlens: num_seqs + 1 entries")
        _need(max_len is None or max_len >= 0, "max_len: not negative")
        longest = total if max_len is None else int(max_len)
    else:
        n = int(num_seqs) if num_seqs is not None else (q.shape[0] if q.dim() == 4 else 1)
        _need(n >= 1 and total % n == 0, "without cu_seqlens every sequence has as many rows")
        longest = total // n
        _need(max_len is None or max_len == longest, "max_len: rows / num_seqs without cu_seqlens")
    _need(n >= 1, "one sequence at least")
    desc = _LinattnDesc(n, H, d, d, _IO_OF[q.dtype], total, longest, qs, ks, vs, 0)
    return desc, total, n, H, d


def pace_linattn_workspace_bytes(num_seqs: int, num_heads: int, d: int, io: int, total_tokens: int, max_len: int,
                                 backward: bool = False) -> int:
    desc = _LinattnDesc(num_seqs, num_heads, d, d, io, total_tokens, max_len, 0, 0, 0, 0)
    n = ctypes.c_size_t()
    _check("pace_linattn_workspace_bytes", lib.pace_linattn_workspace_bytes(ctypes.byref(desc), int(backward),
                                                                            ctypes.byref(n)))
    return n.value


def _tensors(*named) -> None:
    for name, t in named:
        _need(t is None or (isinstance(t, torch.Tensor) and t.is_cuda), f"{name}: a device tensor")


def _lin_workspace(fn: str, desc, backward: int) -> int:
    size = ctypes.c_size_t()
    _check(fn, lib.pace_linattn_workspace_bytes(ctypes.byref(desc), backward, ctypes.byref(size)))
    return size.value


def pace_linattn_forward(q, k, v, log_decay, o=None, ST=None, num_seqs=None, max_len=None, cu_seqlens=None, S0=None,
                         workspace=None, flags=None, stream=None, need_ST=True):
    """Linear attention with a fixed decay for each head over prompts: returns (o, ST).

    q, k, v: [tokens, H, d] packed prompts (or [N, T, H, d]); log_decay: fp32 [H];
    cu_seqlens: int32 [N + 1], or None for prompts of one length; S0, ST: fp32 [N, H, d, d].  Rows of no sequence
    are left as they are (unset in an o made here).
    """
    num_seqs, max_len = _whole("num_seqs", num_seqs), _whole("max_len", max_len)

    def build():
        _tensors(("q", q), ("k", k), ("v", v), ("log_decay", log_decay), ("o", o), ("ST", ST), ("cu_seqlens", cu_seqlens),
                 ("S0", S0), ("flags", flags))
        desc, total, n, H, d = _linattn(q, k, v, log_decay, num_seqs, max_len, cu_seqlens)
        if o is not None:
            to, desc.o_stride = _rows("o", o, H, d, q)
            _need(to == total, "o: as many rows as q")
        _plain("log_decay", log_decay, (H,), torch.float32, q)
        _plain("cu_seqlens", cu_seqlens, (n + 1,), torch.int32, q)
        _plain("S0", S0, (n, H, d, d), torch.float32, q)
        _plain("ST", ST, (n, H, d, d), torch.float32, q)
        _plain("flags", flags, (1,), torch.int32, q)
        return (desc, ctypes.byref(desc), (n, H, d, d), _lin_workspace("pace_linattn_forward", desc, 0),
                _wants_grad(q, k, v, log_decay, S0))

    _, ref, states, size, grads = _plan(("fwd", _form(q), _form(k), _form(v), _form(log_decay), _form(o), _form(ST),
                                     _form(cu_seqlens), _form(S0), _form(flags), num_seqs, max_len), build)
    if grads:
        _detached("pace_linattn_forward")
    if o is None:
        o = _like(q, stream)
    if ST is None and need_ST:
        ST = _new(states, torch.float32, q, stream) if S0 is None else _like(S0, stream)
    ws = _workspace("pace_linattn_forward", size, workspace, q, stream)
    _run("pace_linattn_forward", lib.pace_linattn_forward, q.get_device(), stream, ref, q.data_ptr(), k.data_ptr(),
         v.data_ptr(), log_decay.data_ptr(), _opt(cu_seqlens), _opt(S0), o.data_ptr(), _opt(ST), _opt(ws), _opt(flags))
    return o, ST


def pace_linattn_backward(q, k, v, log_decay, d_o, dq=None, dk=None, dv=None, dS0=None, num_seqs=None, max_len=None,
                          cu_seqlens=None, S0=None, dST=None, workspace=None, flags=None, stream=None, need_dS0=None):
    """Gradients of pace_linattn_forward: returns (dq, dk, dv, dS0); dS0 is None unless S0 or need_dS0 is given.

    dq, dk, dv have the row strides of q, k, v; those not given are made so (rows of no sequence are left unset).
    """
    num_seqs, max_len = _whole("num_seqs", num_seqs), _whole("max_len", max_len)

    def build():
        _tensors(("q", q), ("k", k), ("v", v), ("log_decay", log_decay), ("d_o", d_o), ("dq", dq), ("dk", dk), ("dv", dv),
                 ("dS0", dS0), ("cu_seqlens", cu_seqlens), ("S0", S0), ("dST", dST), ("flags", flags))
        desc, total, n, H, d = _linattn(q, k, v, log_decay, num_seqs, max_len, cu_seqlens)
        to, desc.o_stride = _rows("d_o", d_o, H, d, q)
        _need(to == total, "d_o: as many rows as q")
        rooms = []               # elements to make a strided gradient in; None: packed
        for name, given, stride in (("dq", dq, desc.q_stride), ("dk", dk, desc.k_stride), ("dv", dv, desc.v_stride)):
            rooms.append(None if stride in (0, H * d) else max(total, 1) * stride)
            if given is not None:
                tg, sg = _rows(name, given, H, d, q)
                _need(tg == total and (total <= 1 or (sg or H * d) == (stride or H * d)), f"{name}: rows as those of {name[1:]}")
        _plain("log_decay", log_decay, (H,), torch.float32, q)
        _plain("cu_seqlens", cu_seqlens, (n + 1,), torch.int32, q)
        _plain("S0", S0, (n, H, d, d), torch.float32, q)
        _plain("dST", dST, (n, H, d, d), torch.float32, q)
        _plain("dS0", dS0, (n, H, d, d), torch.float32, q)
        _plain("flags", flags, (1,), torch.int32, q)
        return (desc, ctypes.byref(desc), (n, H, d, d), rooms, _lin_workspace("pace_linattn_backward", desc, 1),
                _wants_grad(q, k, v, log_decay, S0, d_o, dST))

    _, ref, states, rooms, size, grads = _plan(
        ("bwd", _form(q), _form(k), _form(v), _form(log_decay), _form(d_o), _form(dq), _form(dk), _form(dv), _form(dS0),
         _form(cu_seqlens), _form(S0), _form(dST), _form(flags), num_seqs, max_len), build)
    if grads:
        _detached("pace_linattn_backward")
    made = []
    for given, like, room in ((dq, q, rooms[0]), (dk, k, rooms[1]), (dv, v, rooms[2])):
        if given is None:
            given = (_like(like, stream) if room is None
                     else _new(room, like.dtype, q, stream).as_strided(like.shape, like.stride()))
        made.append(given)
    dq, dk, dv = made
    if dS0 is None and (S0 is not None if need_dS0 is None else need_dS0):
        dS0 = _new(states, torch.float32, q, stream)
    ws = _workspace("pace_linattn_backward", size, workspace, q, stream)
    _run("pace_linattn_backward", lib.pace_linattn_backward, q.get_device(), stream, ref, q.data_ptr(), k.data_ptr(),
         v.data_ptr(), log_decay.data_ptr(), _opt(cu_seqlens), _opt(S0), d_o.data_ptr(), _opt(dST), dq.data_ptr(),
         dk.data_ptr(), dv.data_ptr(), _opt(dS0), _opt(ws), _opt(flags))
    return dq, dk, dv, dS0


def pace_linattn_step(S, q, k, v, log_decay, o=None, stream=None) -> torch.Tensor:
    """One token for each of N sequences: q, k, v [N, H, d]; S fp32 [N, H, d, d] is updated in place; returns o."""

    def build():
        _tensors(("S", S), ("q", q), ("k", k), ("v", v), ("log_decay", log_decay), ("o", o))
        _need(isinstance(q, torch.Tensor) and q.dim() == 3, "q: device tensor [N, H, d]")
        _need(q.dtype in _IO_OF, f"q: bfloat16 or float32, not {q.dtype}")
        n, H, d = q.shape
        strides = []
        for name, t in (("q", q), ("k", k), ("v", v), ("o", o)):
            rows, st = (n, 0) if name == "o" and t is None else _rows(name, t, H, d, q)
            _need(rows == n, f"{name}: {n} rows")
            strides.append(st)
        _need(S is not None and log_decay is not None, "S and log_decay: the states and the heads' log decays")
        _plain("S", S, (n, H, d, d), torch.float32, q)
        _plain("log_decay", log_decay, (H,), torch.float32, q)
        desc = _LinattnDesc(n, H, d, d, _IO_OF[q.dtype], 0, 0, *strides)
        return desc, ctypes.byref(desc), _wants_grad(S, q, k, v, log_decay)

    _, ref, grads = _plan(("step", _form(S), _form(q), _form(k), _form(v), _form(log_decay), _form(o)), build)
    if grads:
        _detached("pace_linattn_step")
    if o is None:
        o = _like(q, stream)
    _run("pace_linattn_step", lib.pace_linattn_step, q.get_device(), stream, ref, S.data_ptr(), q.data_ptr(), k.data_ptr(),
         v.data_ptr(), log_decay.data_ptr(), o.data_ptr())
    return o


def pace_debug_linattn_wait(wait_tries: int, extra_tx_bytes: int) -> None:
    _check("pace_debug_linattn_wait", lib.pace_debug_linattn_wait(int(wait_tries), int(extra_tx_bytes)))


_NORM_OF = {"l2": PACE_NORM_L2, "rms": PACE_NORM_RMS, PACE_NORM_L2: PACE_NORM_L2, PACE_NORM_RMS: PACE_NORM_RMS}


def _norm_kind(norm) -> int:
    try:
        return _NORM_OF[norm]
    except (KeyError, TypeError):                # TypeError: nothing that can be looked up
        raise ValueError(f"norm: 'l2' or 'rms', not {norm!r}") from None


def _qk_norm(q, k, q_weight, k_weight, positions, inv_freq, rotary_dim, interleaved, norm, eps, q_scale):
    """Descriptor (strides of q and k set), the tensor that gives type and device, heads, rows and d."""
    like = q if q is not None else k
    _need(isinstance(like, torch.Tensor) and like.dim() >= 3, "q or k: device tensor [..., heads, d]")
    _need(like.dtype in _IO_OF, f"q, k: bfloat16 or float32, not {like.dtype}")
    d = like.shape[-1]
    heads, rows, strides = [0, 0], [], [0, 0]
    for i, (name, t) in enumerate((("q", q), ("k", k))):
        if t is None:
            continue
        _need(isinstance(t, torch.Tensor) and t.dim() >= 3, f"{name}: [..., heads, d]")
        heads[i] = t.shape[-2]
        n, strides[i] = _rows(name, t, heads[i], d, like)
        rows.append(n)
    _need(len(set(rows)) == 1, "q and k: as many rows")
    half = int(rotary_dim) // 2
    if rotary_dim:
        _need(positions is not None and inv_freq is not None, "positions and inv_freq: given with rotary_dim")
    _need(positions is None or positions.numel() == rows[0], f"positions: {rows[0]} of them")
    _plain("q_weight", q_weight, (d,), torch.float32, like)
    _plain("k_weight", k_weight, (d,), torch.float32, like)
    _plain("positions", positions, () if positions is None else positions.shape, torch.int32, like)
    _plain("inv_freq", inv_freq, (half,), torch.float32, like)
    desc = _QkNormDesc(rows[0], heads[0], heads[1], d, int(rotary_dim), int(bool(interleaved)), norm,
                       _IO_OF[like.dtype], float(eps), float(q_scale), strides[0], strides[1], 0, 0)
    return desc, like, heads, rows[0], d


def pace_qk_norm_rotate(q, k, q_weight=None, k_weight=None, positions=None, inv_freq=None, q_out=None, k_out=None,
                        rotary_dim=0, interleaved=False, norm="rms", eps=1e-6, q_scale=1.0, stream=None):
    """Queries and keys normalised for each head and turned by their position: returns (q_out, k_out).

    q: [tokens, Hq, d], k: [tokens, Hk, d] (either may be None); q_out may be q, k_out may be k.
    """
    rotary_dim, interleaved, norm = _whole("rotary_dim", rotary_dim) or 0, bool(interleaved), _norm_kind(norm)
    eps, q_scale = _number("eps", eps), _number("q_scale", q_scale)

    def build():
        _tensors(("q", q), ("k", k), ("q_weight", q_weight), ("k_weight", k_weight), ("positions", positions),
                 ("inv_freq", inv_freq), ("q_out", q_out), ("k_out", k_out))
        desc, like, heads, rows, d = _qk_norm(q, k, q_weight, k_weight, positions, inv_freq, rotary_dim, interleaved, norm,
                                              eps, q_scale)
        for i, (name, t, x) in enumerate((("q_out", q_out, q), ("k_out", k_out, k))):
            _need(x is not None or t is None, f"{name}: given without its input")
            if t is None:
                continue
            n, st = _rows(name, t, heads[i], d, like)
            _need(n == rows, f"{name}: {rows} rows")
            if i:
                desc.k_out_stride = st
            else:
                desc.q_out_stride = st
        return desc, ctypes.byref(desc), _wants_grad(q, k, q_weight, k_weight)

    _, ref, grads = _plan(("norm", _form(q), _form(k), _form(q_weight), _form(k_weight), _form(positions), _form(inv_freq),
                    _form(q_out), _form(k_out), rotary_dim, interleaved, norm, eps, q_scale), build)
    if grads:
        _detached("pace_qk_norm_rotate")
    if q_out is None and q is not None:
        q_out = _like(q, stream)
    if k_out is None and k is not None:
        k_out = _like(k, stream)
    _run("pace_qk_norm_rotate", lib.pace_qk_norm_rotate, (k if q is None else q).get_device(), stream, ref, _opt(q), _opt(k),
         _opt(q_weight), _opt(k_weight), _opt(positions), _opt(inv_freq), _opt(q_out), _opt(k_out))
    return q_out, k_out


def pace_qk_norm_workspace_bytes(num_tokens: int, num_q_heads: int, num_k_heads: int, head_dim: int, io: int) -> int:
    desc = _QkNormDesc(num_tokens, num_q_heads, num_k_heads, head_dim, 0, 0, PACE_NORM_RMS, io, 1e-6, 1.0, 0, 0, 0, 0)
    n = ctypes.c_size_t()
    _check("pace_qk_norm_workspace_bytes", lib.pace_qk_norm_workspace_bytes(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def pace_qk_norm_rotate_backward(q, k, q_weight, k_weight, positions, inv_freq, d_q_out, d_k_out, dq=None, dk=None,
                                 dq_weight=None, dk_weight=None, rotary_dim=0, interleaved=False, norm="rms", eps=1e-6,
                                 q_scale=1.0, workspace=None, stream=None):
    """Gradients of pace_qk_norm_rotate: returns (dq, dk, dq_weight, dk_weight); a weight's gradient is made where the
    weight is given (or a tensor for it)."""
    rotary_dim, interleaved, norm = _whole("rotary_dim", rotary_dim) or 0, bool(interleaved), _norm_kind(norm)
    eps, q_scale = _number("eps", eps), _number("q_scale", q_scale)

    def build():
        _tensors(("q", q), ("k", k), ("q_weight", q_weight), ("k_weight", k_weight), ("positions", positions),
                 ("inv_freq", inv_freq), ("d_q_out", d_q_out), ("d_k_out", d_k_out), ("dq", dq), ("dk", dk),
                 ("dq_weight", dq_weight), ("dk_weight", dk_weight))
        desc, like, heads, rows, d = _qk_norm(q, k, q_weight, k_weight, positions, inv_freq, rotary_dim, interleaved, norm,
                                              eps, q_scale)
        for i, (x, dy, dx, dw) in enumerate(((q, d_q_out, dq, dq_weight), (k, d_k_out, dk, dk_weight))):
            name = "qk"[i]
            _need((x is None) == (dy is None), f"d_{name}_out: given with {name}")
            if x is None:
                _need(dx is None and dw is None, f"d{name}: given without {name}")
                continue
            n, st = _rows(f"d_{name}_out", dy, heads[i], d, like)
            _need(n == rows and (n <= 1 or st in (0, heads[i] * d)), f"d_{name}_out: {rows} packed rows")
            if dx is not None:
                n, st = _rows(f"d{name}", dx, heads[i], d, like)
                _need(n == rows, f"d{name}: {rows} rows")
                if i:
                    desc.k_out_stride = st
                else:
                    desc.q_out_stride = st
            _plain(f"d{name}_weight", dw, (d,), torch.float32, like)
        size = ctypes.c_size_t()
        _check("pace_qk_norm_rotate_backward", lib.pace_qk_norm_workspace_bytes(ctypes.byref(desc), ctypes.byref(size)))
        return desc, ctypes.byref(desc), size.value, _wants_grad(q, k, q_weight, k_weight, d_q_out, d_k_out)

    _, ref, size, grads = _plan(
        ("normb", _form(q), _form(k), _form(q_weight), _form(k_weight), _form(positions), _form(inv_freq), _form(d_q_out),
         _form(d_k_out), _form(dq), _form(dk), _form(dq_weight), _form(dk_weight), rotary_dim, interleaved, norm, eps,
         q_scale), build)
    if grads:
        _detached("pace_qk_norm_rotate_backward")
    like = q if q is not None else k
    if dq is None and q is not None:
        dq = _like(q, stream)
    if dk is None and k is not None:
        dk = _like(k, stream)
    if dq_weight is None and q is not None and q_weight is not None:
        dq_weight = _like(q_weight, stream)
    if dk_weight is None and k is not None and k_weight is not None:
        dk_weight = _like(k_weight, stream)
    ws = None
    if dq_weight is not None or dk_weight is not None:
        ws = _workspace("pace_qk_norm_rotate_backward", size, workspace, like, stream)
    _run("pace_qk_norm_rotate_backward", lib.pace_qk_norm_rotate_backward, like.get_device(), stream, ref, _opt(q), _opt(k),
         _opt(q_weight), _opt(k_weight), _opt(positions), _opt(inv_freq), _opt(d_q_out), _opt(d_k_out), _opt(dq), _opt(dk),
         _opt(dq_weight), _opt(dk_weight), _opt(ws))
    return dq, dk, dq_weight, dk_weight


def pace_status_string(status: int) -> str:
    return _status_name(status)


def pace_version() -> str:
    return lib.pace_version().decode()


# ---------------------------------------------------------------- pool owner

class PacePool:
    """Allocates a pool's three device regions with torch and binds them.

    ``state``, ``buffer`` and ``aux`` are uint8 device tensors; their layout is
    the one documented in ``include/pace.h``.
    """

    def __init__(self, B: int, H: int, d_k: int, d_v: int, P: int, head_bits: Sequence[int],
                 axis: str = "col", io: str = "bf16", device="cuda", stream=None,
                 buffer_e4m3: bool = False):
        self.B, self.H, self.d_k, self.d_v, self.P = B, H, d_k, d_v, P
        self.buffer_e4m3 = bool(buffer_e4m3)
        self.head_bits = [int(b) for b in head_bits]
        self.axis = PACE_SCALE_COL if axis == "col" else PACE_SCALE_ROW
        self.io = PACE_IO_BF16 if io == "bf16" else PACE_IO_F32
        self.io_torch = torch.bfloat16 if io == "bf16" else torch.float32
        sb, bb, ab = pace_pool_bytes(B, H, d_k, d_v, P, self.axis, self.io, self.head_bits,
                                     int(self.buffer_e4m3))
        self.state = torch.empty(sb, dtype=torch.uint8, device=device)
        self.buffer = torch.zeros(bb, dtype=torch.uint8, device=device)
        self.aux = torch.empty(ab, dtype=torch.uint8, device=device)
        self.handle = pace_init_pool(B, H, d_k, d_v, P, self.axis, self.io, self.head_bits,
                                     self.state, self.buffer, self.aux, stream, int(self.buffer_e4m3))
        self.slot_stride = pace_pool_layout(self.handle, 0)[2]

    def __del__(self):
        h = getattr(self, "handle", None)
        if h and pace_destroy_pool is not None:   # module globals are gone at interpreter exit
            try:
                pace_destroy_pool(h)
            except Exception:
                pass
            self.handle = None

    # layout helpers -----------------------------------------------------
    def record(self, b: int, h: int) -> torch.Tensor:
        """View of head (b, h)'s record (codes then fp16 scales) in the state region."""
        off, nbytes, stride = pace_pool_layout(self.handle, h)
        start = b * stride + off
        return self.state[start:start + nbytes]

    def fill(self) -> torch.Tensor:
        return self.aux[: 4 * self.B * self.H].view(torch.int32).view(self.B, self.H)

    # calls ----------------------------------------------------------------
    def load(self, S: torch.Tensor, stream=None) -> None:
        pace_pool_load(self.handle, S, stream)

    def export(self, S: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        if S is None:
            S = torch.empty(self.B, self.H, self.d_v, self.d_k, dtype=torch.float32,
                            device=self.state.device)
        pace_pool_export(self.handle, S, stream)
        return S

    def decode_step(self, q, k, v, alpha, beta, o=None, stream=None) -> torch.Tensor:
        if o is None:
            o = torch.empty(self.B, self.H, self.d_v, dtype=torch.float32, device=self.state.device)
        pace_decode_step(self.handle, q, k, v, alpha, beta, o, stream)
        return o

    def commit_period(self, stream=None) -> None:
        pace_commit_period(self.handle, stream)

    def decode_step_range(self, slot_begin, slot_count, q, k, v, alpha, beta, o, blocks_per_sm=0,
                          stream=None) -> torch.Tensor:
        pace_decode_step_range(self.handle, slot_begin, slot_count, blocks_per_sm, q, k, v, alpha,
                               beta, o, stream)
        return o

    def prefill(self, q, k, v, alpha, beta, o=None, stream=None) -> Optional[torch.Tensor]:
        """T tokens [T][B][H][d] through the chunked fp32 prefill; returns o."""
        pace_prefill(self.handle, int(q.shape[0]), q, k, v, alpha, beta, o, stream)
        return o

    def window_step(self, q, k, v, alpha, beta, o=None, stream=None) -> torch.Tensor:
        """One pure-write-window step (window length = P) for every head."""
        if getattr(self, "_wscratch", None) is None:
            self._wscratch = torch.empty(pace_window_scratch_bytes(self.handle), dtype=torch.uint8,
                                         device=self.state.device)
        if o is None:
            o = torch.empty(self.B, self.H, self.d_v, dtype=torch.float32, device=self.state.device)
        pace_window_step(self.handle, q, k, v, alpha, beta, o, self._wscratch, stream)
        return o

    def set_commit_engine(self, engine: int) -> None:
        """PACE_COMMIT_MMA (default) or PACE_COMMIT_TCGEN05 for later commits."""
        pace_set_commit_engine(self.handle, engine)

    def set_commit_threshold(self, tau: float) -> None:
        """Adaptive period: a head is committed early once the Frobenius norm of
        its update since the last rounding reaches tau (inf: fixed period)."""
        pace_set_commit_threshold(self.handle, tau)

    def decode_host(self, q, k, v, alpha, beta, o=None, stream=None) -> None:
        """T decode steps (each followed by the commit of full heads) from host
        tensors [T][B][H][d]; outputs land in the host tensor o (fp32
        [T][B][H][d_v], pinned for full speed) once `stream` completes."""
        if getattr(self, "_staging", None) is None:
            self._staging = torch.empty(pace_host_staging_bytes(self.handle), dtype=torch.uint8,
                                        device=self.state.device)
            self._h2d = torch.cuda.Stream(self.state.device)
            self._d2h = torch.cuda.Stream(self.state.device)
        s = stream if stream is not None else torch.cuda.current_stream(self.state.device)
        pace_decode_host(self.handle, int(q.shape[0]), q, k, v, alpha, beta, o, self._staging, s,
                         self._h2d, self._d2h)

    def commit_period_range(self, slot_begin, slot_count, blocks_per_sm=0, stream=None) -> None:
        pace_commit_period_range(self.handle, slot_begin, slot_count, blocks_per_sm, stream)

    def status(self, stream=None) -> int:
        return pace_pool_status(self.handle, stream)

    def clear_status(self, stream=None) -> None:
        pace_pool_clear_status(self.handle, stream)
