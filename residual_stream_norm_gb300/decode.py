"""Python binding of the decode operators (``include/beam_decode.h``): attention over the slot cache
with a shared prefix, eviction by accumulated attention weight, 4-bit matrix-vector products.

The functions carry the C names, check and marshal their arguments, and raise ``BeamError`` on a
non-zero status; they are reached as ``residual_stream_norm_gb300.beam_...``.
"""
from __future__ import annotations

import ctypes
import math

import torch

HEAD_DIM = 128
CACHE_BF16, CACHE_FP8_E4M3 = 0, 1
_SM_SCALE = HEAD_DIM ** -0.5


def declare(so: ctypes.CDLL) -> None:
    """Argument types of the decode entry points."""
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    so.beam_attn_prefix_workspace.argtypes = [i32, i32, i32, i32, i64, i64, i64, i32]
    so.beam_attn_prefix_workspace.restype = i64
    so.beam_attn_prefix_fwd.argtypes = [vp, i64, vp, vp, vp, i64, vp, i64, vp, vp, i64, i32, f32,
                                        f32, vp, i64, vp, i64, i64, vp, i32, i32, i32, i32, i32,
                                        f32, i64, vp, i64, vp]
    so.beam_attn_prefix_fwd.restype = ctypes.c_int
    so.beam_kv_evict_fwd.argtypes = [vp, vp, vp, vp, i64, vp, vp, vp, i64, i64, i64, i64, vp]
    so.beam_kv_evict_fwd.restype = ctypes.c_int
    so.beam_w4_matvec_fwd.argtypes = [vp, i64, vp, i64, vp, vp, vp, i64, i64, i64, i32, vp]
    so.beam_w4_matvec_fwd.restype = ctypes.c_int


_fns: dict = {}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_bf16, _f32, _i32, _i64, _u8 = (torch.bfloat16, torch.float32, torch.int32, torch.int64,
                                torch.uint8)


def _run(fn: str, index: int, stream, *args) -> None:
    f = _fns.get(fn)
    if f is None:
        from . import lib
        f = _fns[fn] = getattr(lib(), fn)
    if stream is None:
        s = _raw_stream(index)
    else:
        s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if index == _current_device():
        st = f(*args, s)
    else:
        with torch.cuda.device(index):
            st = f(*args, s)
    if st != 0:
        from . import BeamError
        raise BeamError(fn, st)


# The functions below test their tensors in one expression, which is all that good arguments cost (a
# tenth of a microsecond an attribute, beside calls of some microseconds); only when it fails do
# these checks find out what to say.

def _check(t, name: str, dtype, shape, index: int, rows: bool = False) -> None:
    """A CUDA tensor of this type and shape on device `index`: contiguous, or (rows) with contiguous
    rows of its last dimension."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda:
        raise TypeError(f"{name}: expected a CUDA {dtype} tensor")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name}: must be on cuda:{index}")
    if not t.is_contiguous() and not (rows and t.stride(-1) == 1):
        raise ValueError(f"{name}: must be contiguous")


def _row_stride(t: torch.Tensor) -> int:
    if t.shape[0] > 1:
        return t.stride(0)
    return max(t.stride(0), math.prod(t.shape[1:]))


def _head_rows(t, name: str):
    """(T, heads, row stride, device) of a [T, heads, 128] bf16 CUDA tensor with contiguous heads; the
    rows may be strided."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or not t.is_cuda:
        raise TypeError(f"{name}: expected a CUDA bfloat16 tensor")
    if t.dim() == 3:
        T, n, d = t.shape
        st = t.stride()
        if d == HEAD_DIM and st[2] == 1 and (n <= 1 or st[1] == HEAD_DIM):
            return T, n, st[0] if T > 1 else max(st[0], n * HEAD_DIM), t.get_device()
    raise ValueError(f"{name}: expected [T, heads, {HEAD_DIM}] with contiguous heads")


def beam_attn_prefix_workspace(B: int, q_len: int, n_q_heads: int, n_kv_heads: int,
                               n_prefix: int, table_width: int, window: int = 0,
                               key_weights: bool = False) -> int:
    """Bytes of workspace ``beam_attn_prefix_fwd`` needs for these sizes (host only)."""
    from . import BeamError, lib
    n = lib().beam_attn_prefix_workspace(B, q_len, n_q_heads, n_kv_heads, n_prefix, table_width,
                                         window, int(key_weights))
    if n < 0:
        raise BeamError("beam_attn_prefix_workspace", n)
    return n


def beam_attn_prefix_fwd(out, q, k_cache, v_cache, prefix_slots, slot_table, suffix_len, workspace,
                         cache_dtype: int = CACHE_BF16, k_scale: float = 1.0, v_scale: float = 1.0,
                         sm_scale: float | None = None, window: int = 0, lse_out=None,
                         key_weight_out=None, key_weight_in=None, stream=None) -> None:
    """Attention of a decode batch over the slot cache, with a prefix that every sequence shares.

    out, q: [B*q_len, n_q, 128] bf16 (row-strided views allowed); k_cache, v_cache
    [num_slots, n_kv, 128] (bf16, or 1-byte elements for CACHE_FP8_E4M3); prefix_slots [P] int64 or
    None; slot_table [B, N] int64 (rows may be strided); suffix_len [B] int32; workspace: a
    contiguous uint8 tensor of at least ``beam_attn_prefix_workspace`` bytes; lse_out
    [B*q_len, n_q] fp32; key_weight_in / key_weight_out [B, N] fp32 (may be one tensor).  sm_scale
    defaults to 1/sqrt(128).  The last q_len entries of a sequence's suffix are its query tokens."""
    T, nq, q_stride, dev = _head_rows(q, "q")
    oT, oq, out_stride, odev = _head_rows(out, "out")
    if oT != T or oq != nq or odev != dev:
        raise ValueError("out must have q's shape and device")
    P = 0 if prefix_slots is None else prefix_slots.numel()
    fp8 = cache_dtype == CACHE_FP8_E4M3
    try:
        B, N = slot_table.shape
        S, n_kv, d = k_cache.shape
        good = (slot_table.dtype is _i64 and slot_table.get_device() == dev and
                (slot_table.is_contiguous() or slot_table.stride(1) == 1) and
                suffix_len.dtype is _i32 and suffix_len.shape == (B,) and
                suffix_len.get_device() == dev and suffix_len.is_contiguous() and
                (P == 0 or (prefix_slots.dtype is _i64 and prefix_slots.get_device() == dev and
                            prefix_slots.is_contiguous() and prefix_slots.dim() == 1)) and
                d == HEAD_DIM and (k_cache.element_size() == 1 if fp8 else
                                   cache_dtype == CACHE_BF16 and k_cache.dtype is _bf16) and
                k_cache.get_device() == dev and k_cache.is_contiguous() and
                v_cache.dtype is k_cache.dtype and v_cache.shape == k_cache.shape and
                v_cache.get_device() == dev and v_cache.is_contiguous() and
                workspace.get_device() == dev and workspace.is_contiguous())
    except (AttributeError, ValueError):
        good = False
    if not good:
        if not isinstance(slot_table, torch.Tensor) or slot_table.dim() != 2:
            raise TypeError("slot_table: expected a CUDA int64 tensor [B, N]")
        B, N = slot_table.shape
        _check(slot_table, "slot_table", _i64, (B, N), dev, rows=True)
        _check(suffix_len, "suffix_len", _i32, (B,), dev)
        if prefix_slots is not None:
            _check(prefix_slots, "prefix_slots", _i64, (P,), dev)
        if cache_dtype not in (CACHE_BF16, CACHE_FP8_E4M3):
            raise ValueError(f"cache_dtype: {cache_dtype}")
        if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 3 or \
                k_cache.shape[2] != HEAD_DIM or \
                (k_cache.element_size() != 1 if fp8 else k_cache.dtype != _bf16):
            raise TypeError(f"k_cache: expected a CUDA [num_slots, n_kv, {HEAD_DIM}] tensor of " +
                            ("bytes" if fp8 else "bfloat16"))
        _check(k_cache, "k_cache", k_cache.dtype, k_cache.shape, dev)
        _check(v_cache, "v_cache", k_cache.dtype, k_cache.shape, dev)
        raise TypeError("workspace: expected a contiguous CUDA tensor on q's device")
    if T % B if B else T:
        raise ValueError(f"q has {T} rows, not a multiple of the {B} sequences")
    lse = w_in = w_out = None
    ws = 0
    if lse_out is not None:
        if not (lse_out.dtype is _f32 and lse_out.shape == (T, nq) and
                lse_out.get_device() == dev and lse_out.is_contiguous()):
            _check(lse_out, "lse_out", _f32, (T, nq), dev)
        lse = lse_out.data_ptr()
    if key_weight_out is not None:
        _check(key_weight_out, "key_weight_out", _f32, (B, N), dev, rows=True)
        w_out, ws = key_weight_out.data_ptr(), _row_stride(key_weight_out)
        if key_weight_in is not None:
            _check(key_weight_in, "key_weight_in", _f32, (B, N), dev, rows=True)
            w_in = key_weight_in.data_ptr()
            if B > 1 and _row_stride(key_weight_in) != ws:
                raise ValueError("key_weight_in and key_weight_out must have the same row stride")
    elif key_weight_in is not None:
        raise ValueError("key_weight_in without key_weight_out")
    _run("beam_attn_prefix_fwd", dev, stream, out.data_ptr(), out_stride, lse, w_in, w_out, ws,
         q.data_ptr(), q_stride, k_cache.data_ptr(), v_cache.data_ptr(), S, cache_dtype, k_scale,
         v_scale, prefix_slots.data_ptr() if P else None, P, slot_table.data_ptr(),
         slot_table.stride(0) if B > 1 else N, N, suffix_len.data_ptr(), B, T // B if B else 1, nq,
         n_kv, HEAD_DIM, _SM_SCALE if sm_scale is None else sm_scale, window, workspace.data_ptr(),
         workspace.nbytes)


def beam_kv_evict_fwd(table_out, len_out, weight_out, freed_out, table_in, len_in, weight_in,
                      budget: int, recent: int = 0, stream=None) -> None:
    """Keep at most `budget` entries of each row of the slot table: the last `recent` and, of the
    older ones, those with the largest accumulated weight.  table_in / table_out [rows, width]
    int64, weight_in / weight_out [rows, width] fp32, len_in / len_out [rows] int32 (each output may
    be its input), freed_out [rows, F >= width - budget] int64 or None if the width is within the
    budget: the slots that left, -1 behind them."""
    F = 0
    try:
        dev, shape = table_in.get_device(), table_in.shape
        rows, width = shape
        good = (dev >= 0 and table_in.dtype is _i64 and table_out.dtype is _i64 and
                weight_in.dtype is _f32 and weight_out.dtype is _f32 and
                len_in.dtype is _i32 and len_out.dtype is _i32 and
                table_out.shape == shape and weight_in.shape == shape and
                weight_out.shape == shape and len_in.shape == (rows,) and
                len_out.shape == (rows,) and
                table_out.get_device() == dev and weight_in.get_device() == dev and
                weight_out.get_device() == dev and len_in.get_device() == dev and
                len_out.get_device() == dev and
                table_in.is_contiguous() and table_out.is_contiguous() and
                weight_in.is_contiguous() and weight_out.is_contiguous() and
                len_in.is_contiguous() and len_out.is_contiguous())
        if good and freed_out is not None:
            n, F = freed_out.shape
            good = (n == rows and freed_out.dtype is _i64 and freed_out.get_device() == dev and
                    freed_out.is_contiguous())
    except (AttributeError, ValueError):
        good = False
    if not good:
        if not isinstance(table_in, torch.Tensor) or table_in.dim() != 2:
            raise TypeError("table_in: expected a CUDA int64 tensor [rows, width]")
        dev = table_in.get_device()
        rows, width = table_in.shape
        for t, nm, dtype, shape in (
                (table_in, "table_in", _i64, (rows, width)),
                (table_out, "table_out", _i64, (rows, width)),
                (weight_in, "weight_in", _f32, (rows, width)),
                (weight_out, "weight_out", _f32, (rows, width)),
                (len_in, "len_in", _i32, (rows,)), (len_out, "len_out", _i32, (rows,))):
            _check(t, nm, dtype, shape, dev)
        F = freed_out.shape[1] if isinstance(freed_out, torch.Tensor) and freed_out.dim() == 2 else 0
        _check(freed_out, "freed_out", _i64, (rows, F), dev)
    _run("beam_kv_evict_fwd", dev, stream, table_out.data_ptr(), len_out.data_ptr(),
         weight_out.data_ptr(), freed_out.data_ptr() if F else None, F, table_in.data_ptr(),
         len_in.data_ptr(), weight_in.data_ptr(), rows, width, budget, recent)


def beam_w4_matvec_fwd(y, x, w, scales, zeros=None, group: int = 128, stream=None) -> None:
    """y [T, N] bf16 = x [T, K] bf16 times the transpose of the 4-bit weights w [N, K/2] uint8 (low
    four bits: the even column), (w - zeros) * scales per `group` columns: scales [N, K/group] bf16,
    zeros [N, K/group] uint8 in 0..15 or None (8).  The rows of x and y may be strided."""
    try:
        dev = x.get_device()
        T, K = x.shape
        N, half = w.shape
        G = K // group if group > 0 else 0
        good = (dev >= 0 and x.dtype is _bf16 and (x.is_contiguous() or x.stride(1) == 1) and
                y.dtype is _bf16 and y.shape == (T, N) and y.get_device() == dev and
                (y.is_contiguous() or y.stride(1) == 1) and
                w.dtype is _u8 and 2 * half == K and w.get_device() == dev and
                w.is_contiguous() and
                scales.dtype is _bf16 and scales.shape == (N, G) and
                scales.get_device() == dev and scales.is_contiguous() and
                (zeros is None or (zeros.dtype is _u8 and zeros.shape == (N, G) and
                                   zeros.get_device() == dev and zeros.is_contiguous())))
    except (AttributeError, ValueError):
        good = False
    if not good:
        if not isinstance(x, torch.Tensor) or x.dim() != 2 or not isinstance(w, torch.Tensor) or \
                w.dim() != 2:
            raise TypeError("x and w: expected CUDA tensors [T, K] and [N, K/2]")
        dev = x.get_device()
        T, K = x.shape
        N = w.shape[0]
        _check(x, "x", _bf16, (T, K), dev, rows=True)
        _check(y, "y", _bf16, (T, N), dev, rows=True)
        if K % 2:
            raise ValueError("x: K must be even")
        _check(w, "w", _u8, (N, K // 2), dev)
        G = K // group if group > 0 else 0
        _check(scales, "scales", _bf16, (N, G), dev)
        _check(zeros, "zeros", _u8, (N, G), dev)
    _run("beam_w4_matvec_fwd", dev, stream, y.data_ptr(), y.stride(0) if T > 1 else N, x.data_ptr(),
         x.stride(0) if T > 1 else K, w.data_ptr(), scales.data_ptr(),
         None if zeros is None else zeros.data_ptr(), T, N, K, group)
