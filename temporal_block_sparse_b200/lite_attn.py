"""Python binding of the LiteAttention C ABI (include/lite_attn.h).

Argument marshalling only: every step of the forward pass runs in the CUDA library
`liblite_attn.so` built next to this file. There is no fallback -- if the library is missing or
cannot be loaded, every call raises.
"""

from __future__ import annotations

import ctypes
import math
import os
import struct
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblite_attn.so")

LITE_OK = 0
LITE_ERR_INVALID_ARG = -1
LITE_ERR_UNSUPPORTED = -2
LITE_ERR_CUDA = -3
LITE_ERR_TIMEOUT = -4
LITE_ERR_CHECK = -5
LITE_ERR_SCRATCH_LIMIT = -6
NOALLOC_SCRATCH_BYTES = 8 << 20

LITE_OPT_WAIT_LIMIT_NS = 1
LITE_OPT_DEBUG_STALL = 2
LITE_OPT_MAX_CTAS = 3

# every exported symbol and its (argtypes, restype)
_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
SIGNATURES = {
    "lite_attn_fwd": ([_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _F, _P], _I),
    "lite_attn_dense": ([_P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _P], _I),
    "lite_mask_to_list": ([_P, _P, _P, _I, _I, _I, _I, _P], _I),
    "lite_schedule": ([_P, _P, _I, _I, _I, _P], _I),
    "lite_mask_geometry": ([_I, _I, ctypes.POINTER(_I), ctypes.POINTER(_I), ctypes.POINTER(_I)], _I),
    "lite_get_device_status": ([_P], _I),
    "lite_status_string": ([_I], ctypes.c_char_p),
    "lite_set_option": ([_I, ctypes.c_longlong], _I),
    "lite_set_kernel_events": ([_P, _P], _I),
    "lite_attn_fwd_noalloc": ([_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _F, _P], _I),
    "lite_attn_fwd_ex": ([_P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _F, _F, _P], _I),
    "lite_attn_dense_ex": ([_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P], _I),
    "lite_lse_merge": ([_P, _P, _I, _P, _P, _I, _I, _I, _I, _P], _I),
    "lite_dropped_mass": ([_P, _P, _P, _P, _I, _I, _I, _P], _I),
    "lite_mask_to_ranges": ([_P, _P, _P, _I, _I, _I, _I, _P], _I),
    "lite_set_cta_timing": ([_P, _I], _I),
    "lite_scratch_pool_bytes": ([ctypes.POINTER(ctypes.c_longlong)], _I),
    "lite_qk_rope": ([ctypes.c_char_p, _P], _I),
    "lite_attn_span": ([ctypes.c_char_p, _P], _I),
    "lite_attn_prefix": ([ctypes.c_char_p, _P], _I),
    "lite_attn_fwd_list": ([_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _F, _P], _I),
}
MAX_MERGE_PARTS = 8

_lib = None


class LiteAttnError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status} ({status_string(status)})")


def load(path: str = LIB_PATH):
    """Load the CUDA library (once). Raises if it is absent: there is no CPU path."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"CUDA library {path} is missing; build it with __graft_entry__.build()")
        lib = ctypes.CDLL(path)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load().lite_status_string(int(status)).decode()


def _check(fn: str, status: int):
    if status != LITE_OK:
        raise LiteAttnError(fn, status)


def _stream_handle(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def lite_mask_geometry(N: int, d: int) -> Tuple[int, int, int]:
    """(tile, T, W) for sequence length N and head dim d."""
    tile, T, W = _I(), _I(), _I()
    _check("lite_mask_geometry", load().lite_mask_geometry(int(N), int(d), ctypes.byref(tile), ctypes.byref(T),
                                                           ctypes.byref(W)))
    return tile.value, T.value, W.value


def _check_bf16(name, t):
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 4:
        raise ValueError(f"{name} must be a contiguous 4-D bf16 CUDA tensor [B, N, H, d]")


def _check_qkv(q, k, v):
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_bf16(name, t)
    if not (q.shape == k.shape == v.shape):
        raise ValueError("q, k, v must have the same shape [B, N, H, d]")
    if not (q.device == k.device == v.device):
        raise ValueError("q, k, v must be on one device")


def _check_qkv_cross(q, k, v):
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_bf16(name, t)
    if k.shape != v.shape or q.shape[0] != k.shape[0] or q.shape[2:] != k.shape[2:]:
        raise ValueError("q [B, Nq, H, d] and k, v [B, Nk, H, d] must agree in B, H and d")
    if not (q.device == k.device == v.device):
        raise ValueError("q, k, v must be on one device")


def _ranges(r, name):
    """README-style range list -> (ctypes int32 array or None, length)."""
    if r is None or len(r) == 0:
        return None, 0
    vals = [int(x) for x in r]
    return (ctypes.c_int32 * len(vals))(*vals), len(vals)


def new_mask(B: int, H: int, N: int, d: int, device=None, Nk: Optional[int] = None) -> torch.Tensor:
    """A fresh (all-live) Skip-Mask, int32 [B, H, Tq, Wk] holding uint32 bit patterns (Nk defaults to N)."""
    _, T, _ = lite_mask_geometry(N, d)
    _, _, W = lite_mask_geometry(N if Nk is None else Nk, d)
    return torch.zeros((B, H, T, W), dtype=torch.int32, device=device or "cuda")


def lite_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, mask_in: Optional[torch.Tensor] = None,
                  mask_out: Optional[torch.Tensor] = None, scale: Optional[float] = None, tau: float = -10.0,
                  o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, return_lse: bool = True,
                  stream=None):
    """One LiteAttention forward (see include/lite_attn.h). Returns (o, lse or None)."""
    _check_qkv(q, k, v)
    B, N, H, d = q.shape
    if o is None:
        o = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _check_fwd_buffers(q, k, o, lse, mask_in, mask_out)
    st = load().lite_attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), _ptr(lse), _ptr(mask_in),
                              _ptr(mask_out), B, H, N, d, float(scale or 0.0), float(tau), _stream_handle(stream))
    _check("lite_attn_fwd", st)
    return o, lse


def lite_attn_dense(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: Optional[float] = None,
                    o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, return_lse: bool = True,
                    stream=None):
    """No-skip forward through the same kernel. Returns (o, lse or None)."""
    _check_qkv(q, k, v)
    B, N, H, d = q.shape
    if o is None:
        o = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _check_outputs(q, o, lse)
    st = load().lite_attn_dense(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), _ptr(lse), B, H, N, d,
                                float(scale or 0.0), _stream_handle(stream))
    _check("lite_attn_dense", st)
    return o, lse


def lite_mask_to_list(mask: Optional[torch.Tensor], B: int, H: int, N: int, d: int, stream=None):
    """Skip-Mask -> (list int16 [B,H,T,T], counts int32 [B,H,T]); list entries past counts are -1."""
    _, T, W = lite_mask_geometry(N, d)
    dev = mask.device if mask is not None else torch.device("cuda")
    lst = torch.full((B, H, T, T), -1, dtype=torch.int16, device=dev)
    counts = torch.empty((B, H, T), dtype=torch.int32, device=dev)
    st = load().lite_mask_to_list(_ptr(mask), lst.data_ptr(), counts.data_ptr(), B, H, N, d, _stream_handle(stream))
    _check("lite_mask_to_list", st)
    return lst, counts


def lite_schedule(counts: torch.Tensor, stream=None) -> torch.Tensor:
    """Work order int32 [B*H*T] from live counts [B, H, T]."""
    if counts.dtype != torch.int32 or not counts.is_contiguous() or counts.dim() != 3:
        raise ValueError("counts must be contiguous int32 [B, H, T]")
    B, H, T = counts.shape
    order = torch.empty(B * H * T, dtype=torch.int32, device=counts.device)
    _check("lite_schedule", load().lite_schedule(counts.data_ptr(), order.data_ptr(), B, H, T, _stream_handle(stream)))
    return order


def lite_get_device_status(stream=None) -> int:
    """Synchronise and read/clear the device status word (0 = ok)."""
    return load().lite_get_device_status(_stream_handle(stream))


def lite_set_option(option: int, value: int):
    _check("lite_set_option", load().lite_set_option(int(option), int(value)))


def lite_set_kernel_events(before: Optional[torch.cuda.Event], after: Optional[torch.cuda.Event]):
    """Record `before`/`after` around the attention kernel of later calls (None, None to stop)."""
    b = before.cuda_event if before is not None else None
    a = after.cuda_event if after is not None else None
    _check("lite_set_kernel_events", load().lite_set_kernel_events(b, a))


def default_scale(d: int) -> float:
    return 1.0 / math.sqrt(d)


def lite_attn_fwd_list(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lst: torch.Tensor, counts: torch.Tensor,
                       mask_out: Optional[torch.Tensor] = None, scale: Optional[float] = None, tau: float = -10.0,
                       o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, return_lse: bool = True,
                       stream=None):
    """Forward pass over caller-supplied Skip-Lists (int16 [B, H, T, T] live key tiles, descending,
    with int32 [B, H, T] counts, as lite_mask_to_list returns them); flags are OR-ed into mask_out
    (see include/lite_attn.h). The list buffer may be larger than [B, H, T, T]: only its first
    B*H*T*T entries are addressed. Returns (o, lse or None)."""
    _check_qkv(q, k, v)
    B, N, H, d = q.shape
    _, T, _ = lite_mask_geometry(N, d)
    if o is None:
        o = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _check_fwd_buffers(q, k, o, lse, None, mask_out)
    if (lst.dtype != torch.int16 or not lst.is_contiguous() or not lst.is_cuda or lst.device != q.device
            or lst.numel() < B * H * T * T):
        raise ValueError("lst must be a contiguous int16 CUDA tensor of at least B*H*T*T entries on q's device")
    if (counts.dtype != torch.int32 or not counts.is_contiguous() or not counts.is_cuda or counts.device != q.device
            or tuple(counts.shape) != (B, H, T)):
        raise ValueError("counts must be a contiguous int32 CUDA tensor [B, H, T] on q's device")
    st = load().lite_attn_fwd_list(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), _ptr(lse), lst.data_ptr(),
                                   counts.data_ptr(), _ptr(mask_out), B, H, N, d, float(scale or 0.0), float(tau),
                                   _stream_handle(stream))
    _check("lite_attn_fwd_list", st)
    return o, lse


def lite_attn_fwd_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                          lse: Optional[torch.Tensor] = None, mask_in: Optional[torch.Tensor] = None,
                          mask_out: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                          tau: float = -10.0, stream=None):
    """lite_attn_fwd for callers that must not allocate device memory (see include/lite_attn.h).

    The library allocates nothing here: the caller passes every output buffer, and the per-call
    scratch sits in the library's fixed 8 MiB device array (layers needing more are refused with
    LITE_ERR_SCRATCH_LIMIT). Calls that overlap on the GPU race on that array.
    """
    _check_qkv(q, k, v)
    B, N, H, d = q.shape
    _check_fwd_buffers(q, k, o, lse, mask_in, mask_out)
    st = load().lite_attn_fwd_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), _ptr(lse),
                                      _ptr(mask_in), _ptr(mask_out), B, H, N, d, float(scale or 0.0), float(tau),
                                      _stream_handle(stream))
    _check("lite_attn_fwd_noalloc", st)
    return o, lse


def _check_masks(*masks, shape=None, device=None):
    """Skip-Masks: contiguous int32 CUDA tensors, of `shape` [B, H, Tq, Wk] and on `device` when given."""
    for m in masks:
        if m is None:
            continue
        if m.dtype != torch.int32 or not m.is_contiguous() or not m.is_cuda:
            raise ValueError("masks must be contiguous int32 CUDA tensors [B, H, Tq, Wk]")
        if shape is not None and tuple(m.shape) != tuple(shape):
            raise ValueError(f"mask shape {tuple(m.shape)} != [B, H, Tq, Wk] = {tuple(shape)}")
        if device is not None and m.device != device:
            raise ValueError("masks must be on the device of q")


def _check_outputs(q: torch.Tensor, o: torch.Tensor, lse: Optional[torch.Tensor]):
    """o: contiguous bf16 shaped like q [B, Nq, H, d]; lse: contiguous fp32 [B, H, Nq]; both on q's device."""
    _check_bf16("o", o)
    if o.shape != q.shape or o.device != q.device:
        raise ValueError("o must have q's shape [B, Nq, H, d] and device")
    if lse is not None:
        B, Nq, H, _ = q.shape
        if (lse.dtype != torch.float32 or not lse.is_contiguous() or not lse.is_cuda or lse.device != q.device
                or tuple(lse.shape) != (B, H, Nq)):
            raise ValueError("lse must be a contiguous fp32 CUDA tensor [B, H, Nq] on q's device")


def _check_fwd_buffers(q, k, o, lse, mask_in, mask_out):
    """Every device buffer of a masked forward call, checked before the C call (the library cannot
    tell a host pointer or a short buffer from a good one)."""
    B, Nq, H, d = q.shape
    _, Tq, _ = lite_mask_geometry(Nq, d)
    _, _, Wk = lite_mask_geometry(k.shape[1], d)
    _check_outputs(q, o, lse)
    _check_masks(mask_in, mask_out, shape=(B, H, Tq, Wk), device=q.device)


def scratch_pool_bytes() -> int:
    """Device memory held by the library's scratch pool on the current device (0 before any pooled call)."""
    v = ctypes.c_longlong(0)
    _check("lite_scratch_pool_bytes", load().lite_scratch_pool_bytes(ctypes.byref(v)))
    return int(v.value)


def lite_attn_fwd_ex(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, mask_in: Optional[torch.Tensor] = None,
                     mask_out: Optional[torch.Tensor] = None, must_do=None, must_skip=None,
                     scale: Optional[float] = None, tau: float = -10.0, o: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None, return_lse: bool = True, stream=None):
    """Partial attention: q [B, Nq, H, d] against k, v [B, Nk, H, d], with README-style must-do /
    must-skip key-token range lists (see include/lite_attn.h). Returns (o, lse or None)."""
    _check_qkv_cross(q, k, v)
    B, Nq, H, d = q.shape
    Nk = k.shape[1]
    if o is None:
        o = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    _check_fwd_buffers(q, k, o, lse, mask_in, mask_out)
    do_arr, n_do = _ranges(must_do, "must_do")
    skip_arr, n_skip = _ranges(must_skip, "must_skip")
    st = load().lite_attn_fwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), _ptr(lse), _ptr(mask_in),
                                 _ptr(mask_out), ctypes.cast(do_arr, _P) if do_arr is not None else None, n_do,
                                 ctypes.cast(skip_arr, _P) if skip_arr is not None else None, n_skip, B, H, Nq, Nk, d,
                                 float(scale or 0.0), float(tau), _stream_handle(stream))
    _check("lite_attn_fwd_ex", st)
    return o, lse


def lite_attn_dense_ex(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: Optional[float] = None,
                       o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, return_lse: bool = True,
                       stream=None):
    """No-skip partial attention, q [B, Nq, H, d] against k, v [B, Nk, H, d]. Returns (o, lse or None)."""
    _check_qkv_cross(q, k, v)
    B, Nq, H, d = q.shape
    Nk = k.shape[1]
    if o is None:
        o = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    _check_outputs(q, o, lse)
    st = load().lite_attn_dense_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), _ptr(lse), B, H, Nq, Nk,
                                   d, float(scale or 0.0), _stream_handle(stream))
    _check("lite_attn_dense_ex", st)
    return o, lse


def lite_lse_merge(parts, o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                   return_lse: bool = True, stream=None):
    """Combine partial attentions [(o_p [B, N, H, d] bf16, lse_p [B, H, N] fp32), ...] over disjoint
    key sets into (o, lse). o / lse may be one of the parts' tensors (in place)."""
    parts = list(parts)
    if not 1 <= len(parts) <= MAX_MERGE_PARTS:
        raise ValueError(f"1 to {MAX_MERGE_PARTS} parts")
    o0 = parts[0][0]
    B, N, H, d = o0.shape
    for op, lp in parts:
        _check_bf16("o_p", op)
        if op.shape != o0.shape:
            raise ValueError("all partial outputs must have one shape [B, N, H, d]")
        if lp.dtype != torch.float32 or not lp.is_contiguous() or tuple(lp.shape) != (B, H, N):
            raise ValueError("lse_p must be contiguous fp32 [B, H, N]")
    if o is None:
        o = torch.empty_like(o0)
    if lse is None and return_lse:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=o0.device)
    outs = (_P * len(parts))(*[op.data_ptr() for op, _ in parts])
    lses = (_P * len(parts))(*[lp.data_ptr() for _, lp in parts])
    st = load().lite_lse_merge(ctypes.cast(outs, _P), ctypes.cast(lses, _P), len(parts), o.data_ptr(), _ptr(lse),
                               B, H, N, d, _stream_handle(stream))
    _check("lite_lse_merge", st)
    return o, lse


def lite_dropped_mass(lse_live: torch.Tensor, lse_full: torch.Tensor, row_mass: Optional[torch.Tensor] = None,
                      stats: Optional[torch.Tensor] = None, stream=None):
    """Per-row softmax mass a Skip-Mask drops, 1 - exp(lse_live - lse_full), for lse tensors
    [B, H, N] fp32 on the GPU. Returns (row_mass or None, stats) with stats a device fp32 [2] tensor
    {largest per-row value, sum over rows}; reading it synchronises."""
    for name, t in (("lse_live", lse_live), ("lse_full", lse_full)):
        if t.dtype != torch.float32 or not t.is_contiguous() or t.dim() != 3:
            raise ValueError(f"{name} must be a contiguous fp32 [B, H, N] tensor")
    if lse_live.shape != lse_full.shape:
        raise ValueError("lse_live and lse_full differ in shape")
    B, H, N = lse_live.shape
    if row_mass is not None and (row_mass.shape != lse_live.shape or row_mass.dtype != torch.float32):
        raise ValueError("row_mass must match the lse tensors")
    if stats is None:
        stats = torch.empty(2, dtype=torch.float32, device=lse_live.device)
    st = load().lite_dropped_mass(lse_live.data_ptr(), lse_full.data_ptr(), _ptr(row_mass), stats.data_ptr(), B, H,
                                  N, _stream_handle(stream))
    _check("lite_dropped_mass", st)
    return row_mass, stats


def lite_mask_to_ranges(mask: Optional[torch.Tensor], B: int, H: int, N: int, d: int, device=None, stream=None):
    """Range-encoded Skip-List of a mask: (ranges int16 [B, H, T, T+1], nruns int32 [B, H, T]); row r
    holds nruns[r] (start, end) pairs of live key-tile runs, highest first (end exclusive)."""
    _, T, _ = lite_mask_geometry(N, d)
    dev = mask.device if mask is not None else (device or "cuda")
    if mask is not None:
        _check_masks(mask)
    ranges = torch.empty((B, H, T, T + 1), dtype=torch.int16, device=dev)
    nruns = torch.empty((B, H, T), dtype=torch.int32, device=dev)
    st = load().lite_mask_to_ranges(_ptr(mask), ranges.data_ptr(), nruns.data_ptr(), B, H, N, d, _stream_handle(stream))
    _check("lite_mask_to_ranges", st)
    return ranges, nruns


LITE_OPT_SCHEDULE = 4
LITE_OPT_PAIR_STRIDE = 5


def lite_set_cta_timing(buf: Optional[torch.Tensor]):
    """Per-CTA {start ns, end ns, tiles} records of every following attention launch go to buf
    (int64 [capacity, 3] on the GPU); None stops recording."""
    if buf is None:
        _check("lite_set_cta_timing", load().lite_set_cta_timing(None, 0))
        return
    if buf.dtype != torch.int64 or buf.dim() != 2 or buf.shape[1] != 3 or not buf.is_contiguous():
        raise ValueError("buf must be a contiguous int64 [capacity, 3] tensor")
    _check("lite_set_cta_timing", load().lite_set_cta_timing(buf.data_ptr(), buf.shape[0]))


# ---- rotary positions, span attention, shared prefixes

LITE_BF16, LITE_FP16, LITE_FP32, LITE_INT32 = 0, 1, 2, 3
_I32, _I64 = ctypes.c_int32, ctypes.c_int64

# lite_rope_args and lite_span_args of include/lite_attn.h, field by field (packed in one call: these
# operators are also used on a few tokens, where the time of the call itself counts)
_ROPE_ARGS = struct.Struct("=4Q12q5Q2qQq10if4x")
_SPAN_ARGS = struct.Struct("=12Q15q9i2f4x")


def _call_on(fn: str, args: bytes, index: int, stream):
    """Calls library function `fn` on `stream` (default: the current stream of device `index`) with that device current."""
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    call = getattr(_lib or load(), fn)
    if index == torch._C._cuda_getDevice():
        st = call(args, handle)
    else:
        with torch.cuda.device(index):
            st = call(args, handle)
    if st != LITE_OK:
        raise LiteAttnError(fn, st)


def _new(like: torch.Tensor, shape, dtype, stream) -> torch.Tensor:
    """An output on the device of `like`, made for work on `stream`: its memory is not handed out again
    before that work is done."""
    if stream is None:
        return like.new_empty(shape) if like.dtype is dtype else like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _check_stream(stream, index: int):
    if stream is not None and stream.device.index != index:
        raise ValueError("stream must be on the device of q")


def _check_rows(name: str, t: torch.Tensor, dtypes, unit: int, index: int, batch_zero: bool = False):
    """A CUDA tensor [B, N, heads, d] of one of `dtypes` on device `index` whose head dimension is
    contiguous and whose other strides are multiples of `unit` elements (16 bytes)."""
    if t.dim() != 4 or not t.is_cuda or t.dtype not in dtypes:
        raise ValueError(f"{name} must be a 4-D CUDA tensor [B, N, heads, d] of type "
                         f"{' or '.join(str(x)[6:] for x in dtypes)}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on the device of q")
    size, stride = t.shape, t.stride()
    if size[3] > 1 and stride[3] != 1:
        raise ValueError(f"{name}: the head dimension must be contiguous")
    for x in range(3):
        if size[x] > 1 and (stride[x] % unit or stride[x] < (0 if x == 0 and batch_zero else 1)):
            raise ValueError(f"{name}: strides must be positive multiples of 16 bytes")
    if t.data_ptr() % 16:
        raise ValueError(f"{name} must be 16-byte aligned")


def _rows(name: str, t: torch.Tensor, dtypes, unit: int, index: int, batch_zero: bool = False):
    """(shape, strides, address) of a tensor that passes _check_rows."""
    size, st, at = t.shape, t.stride(), t.data_ptr()
    # what nearly every call passes; anything else is looked at dimension by dimension
    if not (len(size) == 4 and t.dtype in dtypes and t.get_device() == index >= 0 and st[3] == 1
            and st[0] > 0 and st[1] > 0 and st[2] > 0 and not ((st[0] | st[1] | st[2]) & (unit - 1)) and not at & 15):
        _check_rows(name, t, dtypes, unit, index, batch_zero)
    return size, st, at


_BF16 = (torch.bfloat16,)


def _rows3(name: str, t: torch.Tensor, index: int):
    """_rows for a bf16 tensor [N, heads, d]: as if it had a batch dimension of one entry."""
    size, st, at = t.shape, t.stride(), t.data_ptr()
    if not (t.dtype is torch.bfloat16 and t.get_device() == index >= 0 and st[2] == 1 and st[0] > 0 and st[1] > 0
            and not ((st[0] | st[1]) & 7) and not at & 15):
        _check_rows(name, t[None], _BF16, 8, index)
    return (1, *size), (0, *st), at


class RopePlan:
    """Frequencies of a rotary embedding over several axes (host data; made once).

    dims: dimensions of the head that each axis turns, e.g. (44, 42, 42) for frame, row and column at
    d = 128 (workload.axis_split); each even. Pairs beyond their sum are left as they are when
    `head_dim` is larger. Pair i of an axis with D dims has frequency theta ** (-2 i / D).
    pairing: "interleaved" turns elements (2p, 2p + 1) together, "half" elements (p, p + d/2).
    freqs: frequencies of all pairs, in order, to use instead (d/2 numbers; scaled or sectioned variants).
    """

    def __init__(self, dims, theta: float = 10000.0, pairing: str = "interleaved", head_dim: Optional[int] = None,
                 freqs=None):
        dims = tuple(int(x) for x in dims)
        if not 1 <= len(dims) <= 4 or any(x < 0 or x % 2 for x in dims):
            raise ValueError("dims: one to four even, non-negative numbers")
        if pairing not in ("interleaved", "half"):
            raise ValueError("pairing must be 'interleaved' or 'half'")
        d = sum(dims) if head_dim is None else int(head_dim)
        if d not in (64, 128) or sum(dims) > d:
            raise ValueError("the head dimension must be 64 or 128 and hold the sum of dims")
        if not (theta > 0.0 and math.isfinite(theta)):
            raise ValueError("theta must be a positive number")
        self.dims, self.theta, self.pairing, self.d = dims, float(theta), pairing, d
        axis = [a for a, x in enumerate(dims) for _ in range(x // 2)]
        freq = [theta ** (-2.0 * i / x) for x in dims for i in range(x // 2)]
        spare = d // 2 - len(axis)
        axis, freq = axis + [0] * spare, freq + [0.0] * spare
        if freqs is not None:
            freq = [float(x) for x in freqs]
            if len(freq) != d // 2 or not all(math.isfinite(x) for x in freq):
                raise ValueError(f"freqs: {d // 2} finite numbers")
        self.axis, self.freq = axis, freq
        self._axis = (_I32 * len(axis))(*axis)
        self._freq = (ctypes.c_double * len(freq))(*freq)
        self._axis_at, self._freq_at = ctypes.addressof(self._axis), ctypes.addressof(self._freq)
        self._halves = int(pairing == "half")


_POS_TYPES = {torch.float32: LITE_FP32, torch.int32: LITE_INT32}
_ROPE_TYPES = {torch.bfloat16: LITE_BF16, torch.float16: LITE_FP16, torch.float32: LITE_FP32}


def _check_weight(name: str, w: torch.Tensor, sizes, index: int):
    if (w.dtype != torch.float32 or not w.is_contiguous() or w.get_device() != index or w.dim() != 1
            or w.numel() not in sizes or w.data_ptr() % 16):
        raise ValueError(f"{name} must be a contiguous, 16-byte aligned fp32 tensor of "
                         f"{' or '.join(str(x) for x in sizes)} elements on the device of q")


def lite_qk_rope(q: torch.Tensor, k: Optional[torch.Tensor], plan: RopePlan, grid=None, start: int = 0,
                 pos: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, q_out: Optional[torch.Tensor] = None,
                 k_out: Optional[torch.Tensor] = None, stream=None):
    """RMS norm (with weights) and rotary positions of q [B, N, H, d] and k [B, N, Hk, d] or None
    (bf16, fp16 or fp32, any strides that are multiples of 16 bytes, e.g. slices of a fused
    projection). Returns (q_out, k_out), bf16.

    Positions: token n is cell start + n of the row-major `grid` (one size per axis of the plan), or
    `pos` [axes, N] or [B, axes, N] (fp32 or int32) gives them. Weights of d elements norm every head by
    itself, weights of heads * d elements norm the token's whole row. q_out / k_out may be given (a
    slice of a key cache, or q / k themselves for bf16 in place).
    """
    dev = q.get_device()
    dtype = q.dtype
    if dtype not in _ROPE_TYPES:
        raise ValueError("q must be bf16, fp16 or fp32")
    types, unit = (dtype,), 4 if dtype == torch.float32 else 8
    (B, N, H, d), qs, q_at = _rows("q", q, types, unit, dev)
    if stream is not None:
        _check_stream(stream, dev)
    if plan.d != d:
        raise ValueError(f"the plan is for head dimension {plan.d}, q has {d}")
    Hk, ks, k_at = 0, (0, 0, 0, 0), 0
    if k is not None:
        k_size, ks, k_at = _rows("k", k, types, unit, dev)
        Hk = k_size[2]
        if k_size != (B, N, Hk, d):
            raise ValueError("q [B, N, H, d] and k [B, N, Hk, d] must agree in B, N and d")
    if (pos is None) == (grid is None):
        raise ValueError("give either grid or pos")
    axes = len(plan.dims)
    cells, pos_at, pos_type, pos_b, pos_a = 0, 0, 0, 0, 0
    if pos is None:
        grid, start = tuple(map(int, grid)), int(start)
        if len(grid) != axes or min(grid) <= 0 or max(grid) >= 1 << 63:
            raise ValueError(f"grid: {axes} positive sizes")
        if not 0 <= start <= math.prod(grid) - N or start >= 1 << 62:
            raise ValueError("tokens start .. start + N - 1 must lie in the grid")
        sizes = (_I64 * axes)(*grid)
        cells = ctypes.addressof(sizes)
    else:
        if start:
            raise ValueError("start belongs to grid")
        size, pos_dtype = pos.shape, pos.dtype
        if (pos_dtype not in _POS_TYPES or pos.get_device() != dev or not pos.is_contiguous()
                or size[-2:] != (axes, N) or len(size) > 3 or (len(size) == 3 and size[0] not in (1, B))):
            raise ValueError(f"pos must be a contiguous fp32 or int32 tensor [{axes}, N] or [B, {axes}, N] on the device of q")
        pos_at, pos_type = pos.data_ptr(), _POS_TYPES[pos_dtype]
        pos_a, pos_b = N, axes * N if len(size) == 3 and size[0] > 1 else 0
    if k is not None and (q_weight is None) != (k_weight is None):
        raise ValueError("q_weight and k_weight go together")
    if k is None and (k_weight is not None or k_out is not None):
        raise ValueError("k_weight and k_out need k")
    norm, eps, qw_at, kw_at = 0, float(eps), 0, 0
    if q_weight is not None:
        _check_weight("q_weight", q_weight, (d, H * d), dev)
        rows = q_weight.numel() != d
        if k is not None:
            _check_weight("k_weight", k_weight, (d, Hk * d), dev)
            # (with one head the two norms are the same: the other tensor decides)
            rows = rows or k_weight.numel() != d
            if rows and (q_weight.numel() != H * d or k_weight.numel() != Hk * d):
                raise ValueError("q_weight and k_weight must both be per head or both per row")
            kw_at = k_weight.data_ptr()
        norm, qw_at = 2 if rows else 1, q_weight.data_ptr()
        if not 0.0 <= eps < math.inf:
            raise ValueError("eps must be a non-negative number")
    if q_out is None:
        q_out = _new(q, (B, N, H, d), torch.bfloat16, stream)
        qos, qo_at = (N * H * d, H * d, d), q_out.data_ptr()
    else:
        qo_size, qos, qo_at = _rows("q_out", q_out, _BF16, 8, dev)
        if qo_size != q.shape:
            raise ValueError("q_out must have q's shape")
    kos, ko_at = ks, 0
    if k is not None:
        if k_out is None:
            k_out = _new(q, (B, N, Hk, d), torch.bfloat16, stream)
            kos, ko_at = (N * Hk * d, Hk * d, d), k_out.data_ptr()
        else:
            ko_size, kos, ko_at = _rows("k_out", k_out, _BF16, 8, dev)
            if ko_size != k_size:
                raise ValueError("k_out must have k's shape")
    args = _ROPE_ARGS.pack(q_at, k_at, qo_at, ko_at, qs[0], qs[1], qs[2], ks[0], ks[1], ks[2], qos[0], qos[1], qos[2],
                           kos[0], kos[1], kos[2], qw_at, kw_at, plan._freq_at, plan._axis_at, pos_at, pos_b, pos_a,
                           cells, start, _ROPE_TYPES[dtype], pos_type, norm, plan._halves, axes, B, N, H, Hk, d, eps)
    _call_on("lite_qk_rope", args, dev, stream)
    return q_out, k_out


def _span_call(fn: str, q, k, v, k_prefix, v_prefix, spans, scale, cap, slopes, q_pos, k_pos, prefix_pos, o, lse,
               return_lse, stream):
    dev = q.get_device()
    (B, Nq, H, d), qs, q_at = _rows("q", q, _BF16, 8, dev, True)
    k_size, ks, k_at = _rows("k", k, _BF16, 8, dev, True)
    v_size, vs, v_at = _rows("v", v, _BF16, 8, dev, True)
    if stream is not None:
        _check_stream(stream, dev)
    _, Nk, Hk, _ = k_size
    if k_size != v_size or k_size[0] != B or k_size[3] != d:
        raise ValueError("q [B, Nq, H, d] and k, v [B, Nk, Hk, d] must agree in B and d, k and v in shape")
    if Hk == 0 or H % Hk:
        raise ValueError("the heads of k must divide the heads of q")
    Np, kps, vps, kp_at, vp_at = 0, (0, 0, 0, 0), (0, 0, 0, 0), 0, 0
    if k_prefix is not None:
        if k_prefix.dim() == 3 and v_prefix.dim() == 3:
            kp_size, kps, kp_at = _rows3("k_prefix", k_prefix, dev)
            vp_size, vps, vp_at = _rows3("v_prefix", v_prefix, dev)
        else:
            kp_size, kps, kp_at = _rows("k_prefix", k_prefix, _BF16, 8, dev)
            vp_size, vps, vp_at = _rows("v_prefix", v_prefix, _BF16, 8, dev)
        Np = kp_size[1]
        if kp_size != vp_size or kp_size != (1, Np, Hk, d):
            raise ValueError("k_prefix and v_prefix must be [Np, Hk, d] with the heads and head dimension of k")
    spans_at, span_batches = 0, 1
    if spans is not None:
        size = spans.shape
        if (spans.dtype != torch.int32 or spans.get_device() != dev or not spans.is_contiguous()
                or size[-2:] != (Nq, 2) or len(size) > 3 or (len(size) == 3 and size[0] not in (1, B))):
            raise ValueError("spans must be a contiguous int32 tensor [Nq, 2] or [B, Nq, 2] on the device of q")
        spans_at, span_batches = spans.data_ptr(), size[0] if len(size) == 3 else 1
    cap = float(cap or 0.0)
    if not 0.0 <= cap < math.inf:
        raise ValueError("cap must be a non-negative number (0: no cap)")
    slopes_at, pos_at, pos_batches, pp_at = 0, [0, 0], 1, 0
    if slopes is not None:
        if slopes.dtype != torch.float32 or not slopes.is_contiguous() or slopes.get_device() != dev or slopes.shape != (H,):
            raise ValueError("slopes must be a contiguous fp32 tensor [H] on the device of q")
        slopes_at = slopes.data_ptr()
        for x, (name, t, n) in enumerate((("q_pos", q_pos, Nq), ("k_pos", k_pos, Nk))):
            if t is None:
                continue
            if (t.dtype != torch.float32 or not t.is_contiguous() or t.get_device() != dev
                    or tuple(t.shape) not in ((n,), (1, n), (B, n))):
                raise ValueError(f"{name} must be a contiguous fp32 tensor [N] or [B, N] on the device of q")
            batches = t.shape[0] if t.dim() == 2 else 1
            if q_pos is not None and k_pos is not None and batches != (q_pos.shape[0] if q_pos.dim() == 2 else 1):
                raise ValueError("q_pos and k_pos must both be for one or both for all batch entries")
            pos_batches, pos_at[x] = batches, t.data_ptr()
        if prefix_pos is not None:
            if (prefix_pos.dtype != torch.float32 or not prefix_pos.is_contiguous() or prefix_pos.get_device() != dev
                    or tuple(prefix_pos.shape) != (Np,)):
                raise ValueError("prefix_pos must be a contiguous fp32 tensor [Np] on the device of q")
            pp_at = prefix_pos.data_ptr()
    elif q_pos is not None or k_pos is not None or prefix_pos is not None:
        raise ValueError("positions belong to slopes")
    given = o is not None or lse is not None
    if o is None:
        o = _new(q, (B, Nq, H, d), torch.bfloat16, stream)
    if lse is None and return_lse:
        lse = _new(q, (B, H, Nq), torch.float32, stream)
    if given:
        _check_outputs(q, o, lse)
    args = _SPAN_ARGS.pack(q_at, k_at, v_at, kp_at, vp_at, o.data_ptr(), 0 if lse is None else lse.data_ptr(), spans_at,
                           slopes_at, pos_at[0], pos_at[1], pp_at, qs[0], qs[1], qs[2], ks[0], ks[1], ks[2], vs[0],
                           vs[1], vs[2], kps[0], kps[1], kps[2], vps[0], vps[1], vps[2], B, Nq, Nk, Np, H, Hk, d,
                           span_batches, pos_batches, float(scale or 0.0), cap)
    _call_on(fn, args, dev, stream)
    return o, lse


def lite_attn_span(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, spans: Optional[torch.Tensor] = None,
                   scale: Optional[float] = None, cap: float = 0.0, slopes: Optional[torch.Tensor] = None,
                   q_pos: Optional[torch.Tensor] = None, k_pos: Optional[torch.Tensor] = None,
                   o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, return_lse: bool = True,
                   stream=None):
    """Attention of q [B, Nq, H, d] over k, v [B, Nk, Hk, d] in which row n sees the keys spans[.., n, 0]
    <= m < spans[.., n, 1] (int32 [Nq, 2] or [B, Nq, 2]; None: all; spans.py makes the usual tables),
    with scores capped by cap * tanh(s / cap) and lowered by slopes[h] * |q_pos - k_pos| where given
    (see include/lite_attn.h). q, k and v may be strided views. Returns (o, lse or None)."""
    return _span_call("lite_attn_span", q, k, v, None, None, spans, scale, cap, slopes, q_pos, k_pos, None, o, lse,
                      return_lse, stream)


def lite_attn_prefix(q: torch.Tensor, k_prefix: torch.Tensor, v_prefix: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                     spans: Optional[torch.Tensor] = None, scale: Optional[float] = None, cap: float = 0.0,
                     slopes: Optional[torch.Tensor] = None, q_pos: Optional[torch.Tensor] = None,
                     k_pos: Optional[torch.Tensor] = None, prefix_pos: Optional[torch.Tensor] = None,
                     o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, return_lse: bool = True,
                     stream=None):
    """lite_attn_span for a batch whose sequences share a prefix: every row also sees all keys of
    k_prefix, v_prefix [Np, Hk, d], which are stored, and where rows are few read, once for the batch.
    spans counts the own keys k, v [B, Nk, Hk, d]. Np or Nk may be 0. Returns (o, lse or None)."""
    return _span_call("lite_attn_prefix", q, k, v, k_prefix, v_prefix, spans, scale, cap, slopes, q_pos, k_pos,
                      prefix_pos, o, lse, return_lse, stream)
