"""Python binding of libattn.so (argument marshalling only).

Every step of the attention path runs in the library's CUDA kernels; this
module converts torch tensors into the pointers, sizes and cache
descriptors that the C ABI (include/attn_decode.h) takes, and turns
non-zero status codes into exceptions.  PyTorch supplies device memory
(including the split-K workspace) and the current stream.  With stream= the
call runs there, and what it allocates belongs there; its inputs have to be
ready for that stream, and the caller waits for it before using the outputs
on another.  There is no CPU fallback: if libattn.so has not been built,
importing the library fails.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libattn.so")

ATTN_OK = 0
ATTN_ERR_INVALID_ARG = 1
ATTN_ERR_UNSUPPORTED = 2
ATTN_ERR_WORKSPACE = 3
ATTN_ERR_CUDA = 4
ATTN_ERR_DEVICE = 5
ATTN_MAX_PARTITIONS = 1024
ATTN_PARTITIONS_BALANCED = -1   # the balanced MLA split (planner request; num_partitions 0)
ATTN_PARTITIONS_TILE_PAIR = -2  # the tile path with two Q tiles per CTA pair

_STATUS_NAMES = {
    ATTN_ERR_INVALID_ARG: "ATTN_ERR_INVALID_ARG",
    ATTN_ERR_UNSUPPORTED: "ATTN_ERR_UNSUPPORTED",
    ATTN_ERR_WORKSPACE: "ATTN_ERR_WORKSPACE",
    ATTN_ERR_CUDA: "ATTN_ERR_CUDA",
    ATTN_ERR_DEVICE: "ATTN_ERR_DEVICE",
}


class AttnError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} returned {_STATUS_NAMES.get(status, status)}")
        self.status = status


ATTN_ROPE_SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}


class attn_rope_t(ctypes.Structure):
    _fields_ = [
        ("turns", ctypes.c_void_p),
        ("rot_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("mscale", ctypes.c_float),
        ("reserved", ctypes.c_int32),
    ]


class attn_head_rows_t(ctypes.Structure):
    _fields_ = [
        ("in_", ctypes.c_void_p),
        ("in_row_stride", ctypes.c_int64),
        ("in_head_stride", ctypes.c_int64),
        ("out", ctypes.c_void_p),
        ("out_row_stride", ctypes.c_int64),
        ("out_head_stride", ctypes.c_int64),
        ("norm_weight", ctypes.c_void_p),
        ("norm_eps", ctypes.c_float),
        ("norm_dim", ctypes.c_int32),
        ("num_heads", ctypes.c_int32),
        ("dim", ctypes.c_int32),
        ("rot_start", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class attn_kv_scale_t(ctypes.Structure):
    _fields_ = [
        ("base", ctypes.c_void_p),
        ("page_stride", ctypes.c_int64),
        ("block_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
        ("block_tokens", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class attn_kv_t(ctypes.Structure):
    _fields_ = [
        ("base", ctypes.c_void_p),
        ("page_stride", ctypes.c_int64),
        ("token_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("page_table", ctypes.c_void_p),
        ("max_pages", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


_c = ctypes
_SIGNATURES = {
    "attn_plan_partitions": [_c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_int,
                             _c.c_int, _c.c_int, _c.c_int, _c.POINTER(_c.c_int),
                             _c.POINTER(_c.c_size_t)],
    "attn_decode": [_c.c_void_p, _c.POINTER(attn_kv_t), _c.POINTER(attn_kv_t), _c.c_void_p,
                    _c.c_void_p, _c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_int,
                    _c.c_int, _c.c_float, _c.c_void_p, _c.c_int, _c.c_int, _c.c_void_p,
                    _c.c_size_t, _c.c_void_p, _c.c_void_p, _c.c_void_p],
    "attn_mla_decode": [_c.c_void_p, _c.POINTER(attn_kv_t), _c.c_void_p, _c.c_int, _c.c_int,
                        _c.c_int, _c.c_int, _c.c_int, _c.c_float, _c.c_void_p, _c.c_int,
                        _c.c_void_p, _c.c_size_t, _c.c_void_p, _c.c_void_p, _c.c_void_p],
    "attn_mla_decode_rows": [_c.c_void_p, _c.POINTER(attn_kv_t), _c.c_void_p, _c.c_void_p,
                             _c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_int,
                             _c.c_float, _c.c_void_p, _c.c_int, _c.c_int, _c.c_void_p,
                             _c.c_size_t, _c.c_void_p, _c.c_void_p, _c.c_void_p],
    "attn_mla_decode_sparse": [_c.c_void_p, _c.POINTER(attn_kv_t), _c.c_void_p, _c.c_int,
                               _c.c_void_p, _c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_float,
                               _c.c_void_p, _c.c_int, _c.c_void_p, _c.c_size_t, _c.c_void_p,
                               _c.c_void_p, _c.c_void_p],
    "attn_splitk_reduce": [_c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int, _c.c_int,
                           _c.c_int, _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p],
    "attn_device_error_flags": [_c.POINTER(_c.c_uint), _c.c_int],
    "attn_selftest_wait_timeout": [_c.c_void_p],
    "attn_decode_noalloc": [_c.c_void_p, _c.POINTER(attn_kv_t), _c.POINTER(attn_kv_t),
                            _c.c_void_p, _c.c_void_p, _c.c_int, _c.c_int, _c.c_int, _c.c_int,
                            _c.c_int, _c.c_int, _c.c_int, _c.c_float, _c.c_void_p, _c.c_int,
                            _c.c_int, _c.c_void_p, _c.c_void_p, _c.c_void_p],
    "attn_rope_turns": [_c.c_int, _c.c_double, _c.c_int, _c.c_double, _c.c_double, _c.c_double,
                        _c.c_double, _c.c_void_p, _c.POINTER(_c.c_float)],
    "attn_qk_norm_rope": [_c.c_void_p, _c.c_void_p,
                          _c.c_void_p, _c.c_void_p, _c.c_int, _c.c_void_p],
    "attn_append_kv": [_c.c_void_p, _c.c_void_p,
                       _c.c_void_p, _c.c_void_p, _c.c_void_p,
                       _c.c_void_p, _c.c_void_p, _c.c_void_p, _c.c_void_p,
                       _c.c_int, _c.c_int, _c.c_int, _c.c_void_p],
    "attn_append_kv_fp8": [_c.c_void_p, _c.c_void_p,
                           _c.c_void_p, _c.c_void_p, _c.c_void_p,
                           _c.c_void_p, _c.c_void_p,
                           _c.c_void_p, _c.c_void_p, _c.c_void_p,
                           _c.c_void_p, _c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_void_p],
    "attn_decode_fp8_workspace": [_c.c_int, _c.c_int, _c.c_int, _c.c_int,
                                  _c.POINTER(_c.c_size_t)],
    "attn_decode_fp8": [_c.c_void_p, _c.c_void_p, _c.c_void_p,
                        _c.c_void_p, _c.c_void_p, _c.c_void_p,
                        _c.c_void_p, _c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_int,
                        _c.c_int, _c.c_float, _c.c_void_p, _c.c_int, _c.c_void_p, _c.c_size_t,
                        _c.c_void_p, _c.c_void_p, _c.c_void_p],
}

_lib = None


def lib():
    """The loaded libattn.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "split_flash_decoding_gb300.build.build()")
        handle = ctypes.CDLL(LIB_PATH)
        for name, argtypes in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.argtypes = argtypes
            fn.restype = ctypes.c_int
        _lib = handle
    return _lib


def _check(fn: str, status: int):
    if status != ATTN_OK:
        raise AttnError(fn, status)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream_handle(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


# The entry points that fill a cache, and attention over one held in 8 bits, are
# called once a layer and step with little work each, so their host side is kept
# short: descriptors are packed (0.1 us each; a ctypes structure takes 0.6), shapes
# and strides are asked for once, the stream by its device. 
_pack_head_rows = struct.Struct("@PqqPqqPfiiiii").pack      # attn_head_rows_t
_pack_kv = struct.Struct("@PqqqiiPii").pack                 # attn_kv_t
_pack_kv_scale = struct.Struct("@Pqqqii").pack              # attn_kv_scale_t


def _stream_of(stream, device: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return stream.cuda_stream


# ---------------------------------------------------------------------------
# cache descriptors
# ---------------------------------------------------------------------------

def kv_descriptor(cache: torch.Tensor, page_table: Optional[torch.Tensor] = None,
                  dtype: torch.dtype = torch.bfloat16) -> attn_kv_t:
    """Describe a cache tensor (bf16, or of the given dtype) for the C ABI.

    Paged: cache [num_pages, page_size, num_kv_heads, dim] with page_table
    int32 [batch, max_pages].  Contiguous: cache [batch, capacity,
    num_kv_heads, dim] and page_table None.  The last dimension must be
    contiguous; other strides are taken from the tensor.
    """
    return attn_kv_t(*_kv_fields(cache, page_table, dtype))


def _kv_fields(cache, page_table, dtype):
    if cache.dtype != dtype:
        raise TypeError("cache must be bf16" if dtype == torch.bfloat16 else
                        f"cache must be {dtype}")
    strides = cache.stride()
    if len(strides) != 4 or strides[3] != 1:
        raise ValueError("cache must be 4-D with contiguous channels")
    pages, page_size, _, _ = cache.shape
    if page_table is None:
        return (cache.data_ptr(), *strides[:3], page_size, pages, 0, 0, 0)
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or not page_table.is_contiguous():
        raise ValueError("page_table must be a contiguous int32 [batch, max_pages] tensor")
    return (cache.data_ptr(), *strides[:3], page_size, pages, page_table.data_ptr(),
            page_table.shape[1], 0)


def scale_descriptor(scale: torch.Tensor, cache: torch.Tensor) -> attn_kv_scale_t:
    """Describe the scales of an 8-bit cache [pages, page_size, heads, dim]:
    fp32 [pages, page_size / block_tokens, heads]; strides are taken from the
    tensor."""
    return attn_kv_scale_t(*_scale_fields(scale, cache.shape))


def _scale_fields(scale, cache_shape):
    strides = scale.stride()
    if scale.dtype != torch.float32 or len(strides) != 3:
        raise ValueError("scales must be an fp32 [pages, blocks, heads] tensor")
    blocks = scale.shape[1]
    if (scale.shape != (cache_shape[0], blocks, cache_shape[2]) or blocks == 0 or
            cache_shape[1] % blocks):
        raise ValueError(f"scales {tuple(scale.shape)} do not fit a cache {tuple(cache_shape)}")
    return (scale.data_ptr(), *strides, cache_shape[1] // blocks, 0)


# K and V usually have one layout: the second descriptor then is the first with
# another address.

def _kv_pair(k_cache, v_cache, page_table, dtype):
    k = _kv_fields(k_cache, page_table, dtype)
    if (v_cache.shape == k_cache.shape and v_cache.stride() == k_cache.stride() and
            v_cache.dtype == dtype):
        return _pack_kv(*k), _pack_kv(v_cache.data_ptr(), *k[1:])
    return _pack_kv(*k), _pack_kv(*_kv_fields(v_cache, page_table, dtype))


def _scale_pair(k_scale, v_scale, k_shape, v_shape):
    k = _scale_fields(k_scale, k_shape)
    if (v_shape == k_shape and v_scale.shape == k_scale.shape and
            v_scale.stride() == k_scale.stride() and v_scale.dtype == torch.float32):
        return _pack_kv_scale(*k), _pack_kv_scale(v_scale.data_ptr(), *k[1:])
    return _pack_kv_scale(*k), _pack_kv_scale(*_scale_fields(v_scale, v_shape))


class Rope:
    """A rotation: turns int64 [rot_dim / 2] on the device (rope_turns), the
    pair layout (interleaved: channels 2i and 2i + 1; otherwise i and i +
    rot_dim / 2), the factor of cos and sin and the first rotated channel."""

    def __init__(self, turns: torch.Tensor, *, interleaved: bool = False, mscale: float = 1.0,
                 start: int = 0):
        if turns.dtype != torch.int64 or turns.dim() != 1 or not turns.is_contiguous():
            raise ValueError("turns must be a contiguous int64 [rot_dim / 2] tensor")
        self.turns = turns
        self.start = start
        self.struct = attn_rope_t(turns.data_ptr(), 2 * turns.shape[0], 1 if interleaved else 0,
                                  mscale, 0)
        self.ref = ctypes.byref(self.struct)


def rope_turns(rot_dim: int, theta: float, *, scaling: str = "plain", factor: float = 1.0,
               original_len: float = 0.0, low: Optional[float] = None,
               high: Optional[float] = None, device=None):
    """Frequencies of a rotation: (turns int64 [rot_dim / 2], mscale).

    turns[i] is theta^(-2i / rot_dim) / 2 pi turns per position, scaled for a
    long context, in units of 2^-64.  scaling: "plain"; "linear" (f / factor);
    "ntk" (the base raised to factor^(rot_dim / (rot_dim - 2))); "yarn" and
    "bands" (f / factor for pairs that turn less than `low` times in
    original_len positions, f for those that turn more than `high` times, a
    ramp over the pair index or over the turns in between; low and high
    default to 1 and 32, 1 and 4).  mscale is 0.1 ln(factor) + 1 for "yarn"."""
    if scaling not in ATTN_ROPE_SCALINGS:
        raise ValueError(f"unknown scaling {scaling!r}")
    low = 1.0 if low is None else low
    high = (4.0 if scaling == "bands" else 32.0) if high is None else high
    turns = torch.empty(max(rot_dim // 2, 0), dtype=torch.int64)
    mscale = ctypes.c_float(1.0)
    _check("attn_rope_turns",
           lib().attn_rope_turns(rot_dim, theta, ATTN_ROPE_SCALINGS[scaling], factor, original_len,
                                 low, high, turns.data_ptr(), ctypes.byref(mscale)))
    return turns if device is None else turns.to(device), mscale.value


def _head_rows(x: torch.Tensor, shape, out: Optional[torch.Tensor], norm: Optional[torch.Tensor],
               eps: float, rot_start: int) -> bytes:
    """x (of this shape) as packed attn_head_rows_t."""
    if x.dtype != torch.bfloat16:
        raise TypeError("head rows must be bf16")
    strides = x.stride()
    if len(strides) != 3 or (strides[2] != 1 and shape[2] != 1):
        raise ValueError("head rows must be [rows, heads, dim] with contiguous channels")
    dst = out_row = out_head = 0
    if out is not None:
        out_row, out_head, channel = out.stride()
        if out.dtype != torch.bfloat16 or out.shape != shape or channel != 1:
            raise ValueError("out must be bf16, shaped as the input, with contiguous channels")
        dst = out.data_ptr()
    weight = norm_dim = 0
    if norm is not None:
        if norm.dtype != torch.bfloat16 or norm.dim() != 1 or not norm.is_contiguous():
            raise ValueError("norm weights must be contiguous bf16 [norm_dim]")
        weight, norm_dim = norm.data_ptr(), norm.shape[0]
    return _pack_head_rows(x.data_ptr(), strides[0], strides[1], dst, out_row, out_head, weight, eps,
                           norm_dim, shape[1], shape[2], rot_start, 0)


def _int32(t: Optional[torch.Tensor], n: int, what: str):
    if t is None:
        return None
    if t.dtype not in (torch.int32, torch.uint32) or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 [{n}] tensor")
    return t.data_ptr()


def _on_current_device(first: torch.Tensor, *tensors) -> int:
    """The library works on the current device: refuse tensors from elsewhere.
    Returns the device's index."""
    device = first.get_device()
    if device < 0:
        raise ValueError("every tensor must be on the GPU")
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError("every tensor must be on the GPU, and on the same")
    current = torch.cuda.current_device()
    if device != current:
        raise ValueError(f"the tensors are on cuda:{device}, the current device is cuda:{current}")
    return device


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------

def attn_plan_partitions(batch: int, num_q_rows: int, num_q_heads: int, num_kv_heads: int,
                         head_dim_v: int, max_kv_len: int, requested: int = 0,
                         num_sms: int = 0, max_q_len: int = 1):
    """Returns (num_partitions, workspace_bytes).  max_q_len (rows of the
    longest sequence) lets the library route a multi-row GQA call: the
    few-row fold keeps split-K, longer row runs get (1, 0)."""
    P = ctypes.c_int(0)
    ws = ctypes.c_size_t(0)
    _check("attn_plan_partitions",
           lib().attn_plan_partitions(num_sms, batch, num_q_rows, max_q_len, num_q_heads,
                                      num_kv_heads, head_dim_v, max_kv_len, requested,
                                      ctypes.byref(P), ctypes.byref(ws)))
    return P.value, ws.value


def _empty(shape, dtype: torch.dtype, device: torch.device, stream, returned: bool = True):
    """Memory for a call on `stream` (None: the current one).

    The allocator hands a freed block to the next request of the stream it came
    from, in that stream's order.  So what a call on another stream uses is taken
    there; what it returns may be used on the current stream as well."""
    if stream is None or device.type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    if stream.cuda_stream == current.cuda_stream:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(current)
    return t


def _workspace(nbytes: int, device, workspace: Optional[torch.Tensor], stream):
    if nbytes == 0:
        return None, 0
    if workspace is None:
        workspace = _empty(nbytes, torch.uint8, device, stream, returned=False)
    return workspace, workspace.numel() * workspace.element_size()


def attn_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                kv_len: torch.Tensor, *, group: int, scale: float, max_kv_len: int,
                page_table: Optional[torch.Tensor] = None, sink: Optional[torch.Tensor] = None,
                q_row_offsets: Optional[torch.Tensor] = None, max_q_len: int = 1,
                causal: bool = False, num_partitions: int = 0,
                workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                lse: Optional[torch.Tensor] = None, return_lse: bool = True, stream=None):
    """Attention of q rows against a KV cache through attn_decode.

    q bf16 [rows, num_q_heads, head_dim] (rows = batch for single-token
    decode, else q_row_offsets[-1]); caches as for kv_descriptor; kv_len
    int32/uint32 [batch] on the device; q_row_offsets int32 [batch + 1] on
    the device or None; sink fp32 [num_q_heads] or None.  num_partitions 0
    plans automatically.  The library's planner routes the call (a few rows
    per sequence keep split-K on the decode kernel; longer row runs take the
    tile kernel, which is not split) and sizes the workspace.  Returns
    (out, lse).
    """
    rows, hq, d = q.shape
    batch = kv_len.shape[0]
    if out is None:
        out = _empty((rows, hq, d), torch.bfloat16, q.device, stream)
    if lse is None and return_lse:
        lse = _empty((rows, hq), torch.float32, q.device, stream)
    P, ws_bytes = attn_plan_partitions(batch, rows, hq, hq // group, d, max_kv_len,
                                       num_partitions, max_q_len=max_q_len)
    ws, ws_size = _workspace(ws_bytes, q.device, workspace, stream)
    kd = kv_descriptor(k_cache, page_table)
    vd = kv_descriptor(v_cache, page_table)
    _check("attn_decode",
           lib().attn_decode(q.data_ptr(), ctypes.byref(kd), ctypes.byref(vd), kv_len.data_ptr(),
                             _ptr(q_row_offsets), batch, rows, hq, group, d, max_q_len,
                             max_kv_len, scale, _ptr(sink), 1 if causal else 0, P, _ptr(ws),
                             ws_size, out.data_ptr(), _ptr(lse), _stream_handle(stream)))
    return out, lse


def attn_mla_decode(q: torch.Tensor, kv_cache: torch.Tensor, kv_len: torch.Tensor, *,
                    scale: float, max_kv_len: int, dim_v: int = 512,
                    page_table: Optional[torch.Tensor] = None,
                    sink: Optional[torch.Tensor] = None, num_partitions: int = 0,
                    workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, return_lse: bool = True, stream=None):
    """MLA decode through attn_mla_decode: q bf16 [batch, num_q_heads, 576],
    one-head cache [pages, page_size, 1, 576]; V = K[..., :dim_v].
    num_partitions: 0 = the planner's choice, > 0 = that many key slices per
    row, ATTN_PARTITIONS_BALANCED = the balanced split (as for the _rows and
    _sparse variants)."""
    batch, hq, dqk = q.shape
    if out is None:
        out = _empty((batch, hq, dim_v), torch.bfloat16, q.device, stream)
    if lse is None and return_lse:
        lse = _empty((batch, hq), torch.float32, q.device, stream)
    P, ws_bytes = attn_plan_partitions(batch, batch, hq, 1, dim_v, max_kv_len, num_partitions)
    ws, ws_size = _workspace(ws_bytes, q.device, workspace, stream)
    kd = kv_descriptor(kv_cache, page_table)
    _check("attn_mla_decode",
           lib().attn_mla_decode(q.data_ptr(), ctypes.byref(kd), kv_len.data_ptr(), batch, hq, dqk,
                                 dim_v, max_kv_len, scale, _ptr(sink), P, _ptr(ws), ws_size,
                                 out.data_ptr(), _ptr(lse), _stream_handle(stream)))
    return out, lse


def attn_mla_decode_rows(q: torch.Tensor, kv_cache: torch.Tensor, kv_len: torch.Tensor,
                         q_row_offsets: torch.Tensor, *, scale: float, max_kv_len: int,
                         causal: bool = True, dim_v: int = 512,
                         page_table: Optional[torch.Tensor] = None,
                         sink: Optional[torch.Tensor] = None, num_partitions: int = 0,
                         workspace: Optional[torch.Tensor] = None,
                         out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                         return_lse: bool = True, stream=None):
    """MLA decode of several query rows per sequence (draft tokens) through
    attn_mla_decode_rows: q bf16 [rows, 128, 576]; q_row_offsets int32
    [batch + 1] on the device; row i of n sees keys j <= L - n + i when
    causal."""
    rows, hq, dqk = q.shape
    batch = kv_len.shape[0]
    if q_row_offsets.shape[0] != batch + 1:
        raise ValueError("q_row_offsets must have batch + 1 entries")
    if out is None:
        out = _empty((rows, hq, dim_v), torch.bfloat16, q.device, stream)
    if lse is None and return_lse:
        lse = _empty((rows, hq), torch.float32, q.device, stream)
    P, ws_bytes = attn_plan_partitions(batch, rows, hq, 1, dim_v, max_kv_len, num_partitions)
    ws, ws_size = _workspace(ws_bytes, q.device, workspace, stream)
    kd = kv_descriptor(kv_cache, page_table)
    _check("attn_mla_decode_rows",
           lib().attn_mla_decode_rows(q.data_ptr(), ctypes.byref(kd), kv_len.data_ptr(),
                                      q_row_offsets.data_ptr(), batch, rows, hq, dqk, dim_v,
                                      max_kv_len, scale, _ptr(sink), 1 if causal else 0, P,
                                      _ptr(ws), ws_size, out.data_ptr(), _ptr(lse),
                                      _stream_handle(stream)))
    return out, lse


def attn_mla_decode_sparse(q: torch.Tensor, kv_cache: torch.Tensor, indices: torch.Tensor,
                           topk_lengths: torch.Tensor, *, scale: float, dim_v: int = 512,
                           sink: Optional[torch.Tensor] = None, num_partitions: int = 0,
                           workspace: Optional[torch.Tensor] = None,
                           out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                           return_lse: bool = True, stream=None):
    """Sparse top-k MLA decode through attn_mla_decode_sparse: q bf16
    [batch, num_q_heads, 576]; kv_cache [num_pages, page_size, 1, 576] read as
    rows (row r = slot r % page_size of page r // page_size); indices int32
    [batch, indices_stride] naming each sequence's rows; topk_lengths int32
    [batch] valid entries per row of indices."""
    batch, hq, dqk = q.shape
    if indices.dtype != torch.int32 or indices.dim() != 2 or not indices.is_contiguous():
        raise ValueError("indices must be a contiguous int32 [batch, indices_stride] tensor")
    if indices.shape[0] != batch or topk_lengths.shape[0] != batch:
        raise ValueError("indices and topk_lengths need one row per sequence")
    stride = indices.shape[1]
    if out is None:
        out = _empty((batch, hq, dim_v), torch.bfloat16, q.device, stream)
    if lse is None and return_lse:
        lse = _empty((batch, hq), torch.float32, q.device, stream)
    P, ws_bytes = attn_plan_partitions(batch, batch, hq, 1, dim_v, stride, num_partitions)
    ws, ws_size = _workspace(ws_bytes, q.device, workspace, stream)
    kd = kv_descriptor(kv_cache)
    _check("attn_mla_decode_sparse",
           lib().attn_mla_decode_sparse(q.data_ptr(), ctypes.byref(kd), indices.data_ptr(), stride,
                                        topk_lengths.data_ptr(), batch, hq, dqk, dim_v, scale,
                                        _ptr(sink), P, _ptr(ws), ws_size, out.data_ptr(),
                                        _ptr(lse), _stream_handle(stream)))
    return out, lse


def attn_splitk_reduce(ws_o: torch.Tensor, ws_m: torch.Tensor, ws_l: torch.Tensor, *,
                       sink: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                       lse: Optional[torch.Tensor] = None, stream=None):
    """Merge fp32 partials ws_o [P, rows, Hq, dv], ws_m / ws_l [P, rows, Hq]."""
    P, rows, hq, dv = ws_o.shape
    for t in (ws_o, ws_m, ws_l):
        if t.dtype != torch.float32 or not t.is_contiguous():
            raise ValueError("partials must be contiguous fp32")
    if out is None:
        out = _empty((rows, hq, dv), torch.bfloat16, ws_o.device, stream)
    if lse is None:
        lse = _empty((rows, hq), torch.float32, ws_o.device, stream)
    _check("attn_splitk_reduce",
           lib().attn_splitk_reduce(ws_o.data_ptr(), ws_m.data_ptr(), ws_l.data_ptr(), P, rows,
                                    hq, dv, _ptr(sink), out.data_ptr(), _ptr(lse),
                                    _stream_handle(stream)))
    return out, lse


def attn_decode_noalloc(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                        kv_len: torch.Tensor, *, group: int, scale: float, max_kv_len: int,
                        page_table: Optional[torch.Tensor] = None,
                        sink: Optional[torch.Tensor] = None,
                        q_row_offsets: Optional[torch.Tensor] = None, max_q_len: int = 1,
                        causal: bool = False, num_partitions: int = 0,
                        out: torch.Tensor, lse: Optional[torch.Tensor] = None, stream=None):
    """attn_decode whose split-K scratch is the library's fixed device array,
    for callers that cannot allocate: the caller passes only inputs and
    outputs (out must be preallocated), and the call allocates nothing."""
    rows, hq, d = q.shape
    batch = kv_len.shape[0]
    kd = kv_descriptor(k_cache, page_table)
    vd = kv_descriptor(v_cache, page_table)
    _check("attn_decode_noalloc",
           lib().attn_decode_noalloc(q.data_ptr(), ctypes.byref(kd), ctypes.byref(vd),
                                     kv_len.data_ptr(), _ptr(q_row_offsets), batch, rows, hq,
                                     group, d, max_q_len, max_kv_len, scale, _ptr(sink),
                                     1 if causal else 0, num_partitions, out.data_ptr(),
                                     _ptr(lse), _stream_handle(stream)))
    return out, lse


def attn_qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor] = None,
                      positions: Optional[torch.Tensor] = None, *, rope: Optional[Rope] = None,
                      q_norm: Optional[torch.Tensor] = None,
                      k_norm: Optional[torch.Tensor] = None, eps: float = 1e-6,
                      q_out: Optional[torch.Tensor] = None,
                      k_out: Optional[torch.Tensor] = None, stream=None):
    """Norm and rotation of query and key heads through attn_qk_norm_rope.

    q, k bf16 [rows, heads, dim], any row and head strides; positions int32
    [rows]; q_norm / k_norm bf16 weights of the leading channels to norm, or
    None.  q_out / k_out may be q / k (in place).  Returns (q_out, k_out)."""
    rows = q.shape[0]
    if k is not None and k.shape[0] != rows:
        raise ValueError("q and k must have the same rows")
    if q_out is None:
        q_out = _empty(q.shape, torch.bfloat16, q.device, stream)
    if k_out is None and k is not None:
        k_out = _empty(k.shape, torch.bfloat16, k.device, stream)
    start = 0 if rope is None else rope.start
    qd = _head_rows(q, q.shape, q_out, q_norm, eps, start)
    kd = None if k is None else _head_rows(k, k.shape, k_out, k_norm, eps, start)
    pos = _int32(positions, rows, "positions")
    device = _on_current_device(q, k, q_out, k_out, positions, q_norm, k_norm,
                                None if rope is None else rope.turns)
    _check("attn_qk_norm_rope",
           lib().attn_qk_norm_rope(qd, kd, None if rope is None else rope.ref, pos, rows,
                                   _stream_of(stream, device)))
    return q_out, k_out


def _append_args(k, v, k_cache, v_cache, kv_len, page_table, q, q_out, q_row_offsets, rope,
                 positions, q_norm, k_norm, eps, stream, dtype, *scales):
    k_shape, kc_shape, batch = k.shape, k_cache.shape, kv_len.shape[0]
    rows = k_shape[0]
    if (v is None) != (v_cache is None):
        raise ValueError("v and v_cache go together")
    if k_shape[1:] != kc_shape[2:]:
        raise ValueError(f"rows {tuple(k_shape)} do not fit a cache {tuple(kc_shape)}")
    if page_table is not None and page_table.shape[0] != batch:
        raise ValueError("page_table must have one row per sequence")
    start, rope_ref = (0, None) if rope is None else (rope.start, rope.ref)
    qd = vd = vc = None
    if q is not None:
        q_shape = q.shape
        if q_shape[0] != rows:
            raise ValueError("q, k and v must have the same rows")
        if q_out is None:
            q_out = _empty(q_shape, torch.bfloat16, q.device, stream)
        qd = _head_rows(q, q_shape, q_out, q_norm, eps, start)
    kd = _head_rows(k, k_shape, None, k_norm, eps, start)
    if v is None:
        kc = _pack_kv(*_kv_fields(k_cache, page_table, dtype))
    else:
        v_shape = v.shape
        if (v_shape != k_shape or v_cache.shape != kc_shape) and (
                v_shape[0] != rows or v_shape[1:] != v_cache.shape[2:]):
            raise ValueError(f"rows {tuple(v_shape)} do not fit {rows} rows and a cache "
                             f"{tuple(v_cache.shape)}")
        vd = _head_rows(v, v_shape, None, None, eps, 0)
        kc, vc = _kv_pair(k_cache, v_cache, page_table, dtype)
    head = (qd, kd, vd, rope_ref, _int32(positions, rows, "positions"), kc, vc)
    tail = (_int32(kv_len, batch, "kv_len"), _int32(q_row_offsets, batch + 1, "q_row_offsets"),
            batch, rows)
    device = _on_current_device(k, v, k_cache, v_cache, kv_len, page_table, q, q_out,
                                q_row_offsets, positions, q_norm, k_norm,
                                None if rope is None else rope.turns, *scales)
    return q_out, head, tail, device


def attn_append_kv(k: torch.Tensor, v: Optional[torch.Tensor], k_cache: torch.Tensor,
                   v_cache: Optional[torch.Tensor], kv_len: torch.Tensor, *, max_kv_len: int,
                   page_table: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                   q_out: Optional[torch.Tensor] = None,
                   q_row_offsets: Optional[torch.Tensor] = None, rope: Optional[Rope] = None,
                   positions: Optional[torch.Tensor] = None,
                   q_norm: Optional[torch.Tensor] = None, k_norm: Optional[torch.Tensor] = None,
                   eps: float = 1e-6, stream=None):
    """Store the keys and values of new tokens through attn_append_kv.

    k, v bf16 [rows, num_kv_heads, dim] (v and v_cache None for a cache whose V
    is part of K), q [rows, num_q_heads, dim] or None; caches and page_table as
    for kv_descriptor; kv_len int32 [batch], the new tokens included;
    q_row_offsets int32 [batch + 1] or None (one row per sequence).  k and q
    are normed (q_norm, k_norm) and rotated (rope) on the way.  Returns q_out."""
    q_out, head, tail, device = _append_args(k, v, k_cache, v_cache, kv_len, page_table, q, q_out,
                                             q_row_offsets, rope, positions, q_norm, k_norm, eps,
                                             stream, torch.bfloat16)
    _check("attn_append_kv",
           lib().attn_append_kv(*head, *tail, max_kv_len, _stream_of(stream, device)))
    return q_out


def attn_append_kv_fp8(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor,
                       v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                       kv_len: torch.Tensor, *, max_kv_len: int,
                       max_q_len: Optional[int] = None,
                       page_table: Optional[torch.Tensor] = None,
                       q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                       q_row_offsets: Optional[torch.Tensor] = None,
                       rope: Optional[Rope] = None, positions: Optional[torch.Tensor] = None,
                       q_norm: Optional[torch.Tensor] = None,
                       k_norm: Optional[torch.Tensor] = None, eps: float = 1e-6, stream=None):
    """attn_append_kv into caches of torch.float8_e4m3fn with fp32 scales
    [pages, page_size / block_tokens, num_kv_heads] (attn_append_kv_fp8), head
    dimension 128.  max_q_len bounds the rows of any sequence; by default, with
    q_row_offsets, it is all rows (right, but a call of short runs is faster with its
    own bound).  Returns q_out."""
    q_out, head, tail, device = _append_args(k, v, k_cache, v_cache, kv_len, page_table, q, q_out,
                                             q_row_offsets, rope, positions, q_norm, k_norm, eps,
                                             stream, torch.float8_e4m3fn, k_scale, v_scale)
    if max_q_len is None:
        max_q_len = 1 if q_row_offsets is None else max(k.shape[0], 1)
    _check("attn_append_kv_fp8",
           lib().attn_append_kv_fp8(*head, *_scale_pair(k_scale, v_scale, k_cache.shape,
                                                       v_cache.shape), *tail,
                                    max_q_len, max_kv_len, _stream_of(stream, device)))
    return q_out


@functools.lru_cache(maxsize=1024)
def _fp8_workspace(device: int, batch: int, num_q_heads: int, group: int) -> int:
    return attn_decode_fp8_workspace(batch, num_q_heads, group)


def attn_decode_fp8_workspace(batch: int, num_q_heads: int, group: int, num_sms: int = 0) -> int:
    """Bytes of workspace that attn_decode_fp8 needs."""
    n = ctypes.c_size_t(0)
    _check("attn_decode_fp8_workspace",
           lib().attn_decode_fp8_workspace(num_sms, batch, num_q_heads, group, ctypes.byref(n)))
    return n.value


def attn_decode_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    k_scale: torch.Tensor, v_scale: torch.Tensor, kv_len: torch.Tensor, *,
                    group: int, scale: float, max_kv_len: int,
                    page_table: Optional[torch.Tensor] = None,
                    sink: Optional[torch.Tensor] = None,
                    q_row_offsets: Optional[torch.Tensor] = None,
                    max_q_len: Optional[int] = None,
                    causal: bool = False, workspace: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    return_lse: bool = True, stream=None):
    """Decode attention over caches of torch.float8_e4m3fn with fp32 scales
    [pages, page_size / block_tokens, num_kv_heads] through attn_decode_fp8:
    one row, or a few (max_q_len * group <= 16), per sequence, head dimension
    128; everything else as for attn_decode.  max_q_len is by default, with
    q_row_offsets, the most that a call may have.  Returns (out, lse)."""
    rows, hq, d = q.shape
    batch = kv_len.shape[0]
    kd, vd = _kv_pair(k_cache, v_cache, page_table, torch.float8_e4m3fn)
    k_shape, v_shape = k_cache.shape, v_cache.shape
    ks, vs = _scale_pair(k_scale, v_scale, k_shape, v_shape)
    if q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise ValueError("q must be contiguous bf16 [rows, num_q_heads, 128]")
    if k_shape[2:] != v_shape[2:] or k_shape[2] * group != hq or k_shape[3] != d:
        raise ValueError(f"{hq} query heads of {d} in groups of {group} do not fit caches "
                         f"{tuple(k_shape)} and {tuple(v_shape)}")
    if page_table is not None and page_table.shape[0] != batch:
        raise ValueError("page_table must have one row per sequence")
    lens = _int32(kv_len, batch, "kv_len")
    offs = _int32(q_row_offsets, batch + 1, "q_row_offsets")
    if sink is not None and (sink.dtype != torch.float32 or sink.shape != (hq,) or
                             not sink.is_contiguous()):
        raise ValueError("sink must be contiguous fp32 [num_q_heads]")
    if out is None:
        out = _empty((rows, hq, d), torch.bfloat16, q.device, stream)
    elif out.dtype != torch.bfloat16 or out.shape != q.shape or not out.is_contiguous():
        raise ValueError("out must be contiguous bf16, shaped as q")
    if lse is None and return_lse:
        lse = _empty((rows, hq), torch.float32, q.device, stream)
    elif lse is not None and (lse.dtype != torch.float32 or lse.shape != (rows, hq) or
                              not lse.is_contiguous()):
        raise ValueError("lse must be contiguous fp32 [rows, num_q_heads]")
    if max_q_len is None:
        max_q_len = 1 if q_row_offsets is None or group < 1 else max(min(rows, 16 // group), 1)
    device = _on_current_device(q, k_cache, v_cache, k_scale, v_scale, kv_len, page_table, sink,
                                q_row_offsets, workspace, out, lse)
    need = 0 if max_kv_len <= 128 else _fp8_workspace(device, batch, hq, group)
    ws, ws_size = _workspace(need, q.device, workspace, stream)
    _check("attn_decode_fp8",
           lib().attn_decode_fp8(q.data_ptr(), kd, vd, ks, vs, lens, offs, batch, rows, hq, group,
                                 d, max_q_len, max_kv_len, scale, _ptr(sink),
                                 1 if causal else 0, _ptr(ws), ws_size, out.data_ptr(), _ptr(lse),
                                 _stream_of(stream, device)))
    return out, lse


def attn_selftest_wait_timeout(stream=None) -> None:
    """Failure-path check: one kernel whose bounded wait on a barrier nothing
    arrives on gives up after its time limit and sets bit 0 of the device
    error word (read it with attn_device_error_flags)."""
    _check("attn_selftest_wait_timeout", lib().attn_selftest_wait_timeout(_stream_handle(stream)))


def attn_device_error_flags(clear: bool = True) -> int:
    flags = ctypes.c_uint(0)
    _check("attn_device_error_flags", lib().attn_device_error_flags(ctypes.byref(flags),
                                                                    1 if clear else 0))
    return flags.value
