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


def _run(fn: str, index: int, stream, *args) -> None:
    f = _fns.get(fn)
    if f is None:
        from . import lib
        f = _fns[fn] = getattr(lib(), fn)
    if stream is None:
        s = torch._C._cuda_getCurrentRawStream(index)
    else:
        s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if index == torch._C._cuda_getDevice():
        st = f(*args, s)
    else:
        with torch.cuda.device(index):
            st = f(*args, s)
    if st != 0:
        from . import BeamError
        raise BeamError(fn, st)


def _check(t, name: str, dtype, shape, index: int, rows: bool = False) -> None:
    """A CUDA tensor of this type and shape on device `index`: contiguous, or (rows) with contiguous
    rows of its last dimension.  The first test is all that a good argument costs."""
    try:
        if t.dtype is dtype and t.get_device() == index and t.shape == shape and \
                (t.is_contiguous() or (rows and t.stride(-1) == 1)):
            return
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda:
        raise TypeError(f"{name}: expected a CUDA {dtype} tensor")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name}: must be on cuda:{index}")
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
    if (oT, oq, odev) != (T, nq, dev):
        raise ValueError("out must have q's shape and device")
    if not isinstance(suffix_len, torch.Tensor) or not isinstance(slot_table, torch.Tensor) or \
            slot_table.dim() != 2:
        raise TypeError("suffix_len and slot_table: expected CUDA tensors [B] int32 and [B, N] int64")
    B, N = slot_table.shape
    _check(suffix_len, "suffix_len", torch.int32, (B,), dev)
    _check(slot_table, "slot_table", torch.int64, (B, N), dev, rows=True)
    if T % B if B else T:
        raise ValueError(f"q has {T} rows, not a multiple of the {B} sequences")
    P = 0
    if prefix_slots is not None:
        P = prefix_slots.numel() if isinstance(prefix_slots, torch.Tensor) else -1
        _check(prefix_slots, "prefix_slots", torch.int64, (P,), dev)
    if cache_dtype not in (CACHE_BF16, CACHE_FP8_E4M3):
        raise ValueError(f"cache_dtype: {cache_dtype}")
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 3 or k_cache.shape[2] != HEAD_DIM \
            or (k_cache.dtype is not torch.bfloat16 if cache_dtype == CACHE_BF16 else
                k_cache.element_size() != 1):
        raise TypeError(f"k_cache: expected a CUDA [num_slots, n_kv, {HEAD_DIM}] tensor of " +
                        ("bfloat16" if cache_dtype == CACHE_BF16 else "bytes"))
    S, n_kv, _ = k_cache.shape
    _check(k_cache, "k_cache", k_cache.dtype, k_cache.shape, dev)
    _check(v_cache, "v_cache", k_cache.dtype, k_cache.shape, dev)
    if not (isinstance(workspace, torch.Tensor) and workspace.get_device() == dev and
            workspace.is_contiguous()):
        raise TypeError("workspace: expected a contiguous CUDA tensor on q's device")
    lse = w_in = w_out = None
    ws = 0
    if lse_out is not None:
        _check(lse_out, "lse_out", torch.float32, (T, nq), dev)
        lse = lse_out.data_ptr()
    if key_weight_out is not None:
        _check(key_weight_out, "key_weight_out", torch.float32, (B, N), dev, rows=True)
        w_out, ws = key_weight_out.data_ptr(), _row_stride(key_weight_out)
        if key_weight_in is not None:
            _check(key_weight_in, "key_weight_in", torch.float32, (B, N), dev, rows=True)
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
    if not isinstance(table_in, torch.Tensor) or table_in.dim() != 2:
        raise TypeError("table_in: expected a CUDA int64 tensor [rows, width]")
    dev = table_in.get_device()
    rows, width = table_in.shape
    _check(table_in, "table_in", torch.int64, (rows, width), dev)
    _check(table_out, "table_out", torch.int64, (rows, width), dev)
    _check(weight_in, "weight_in", torch.float32, (rows, width), dev)
    _check(weight_out, "weight_out", torch.float32, (rows, width), dev)
    _check(len_in, "len_in", torch.int32, (rows,), dev)
    _check(len_out, "len_out", torch.int32, (rows,), dev)
    F = 0
    if freed_out is not None:
        F = freed_out.shape[1] if isinstance(freed_out, torch.Tensor) and freed_out.dim() == 2 else 0
        _check(freed_out, "freed_out", torch.int64, (rows, F), dev)
    _run("beam_kv_evict_fwd", dev, stream, table_out.data_ptr(), len_out.data_ptr(),
         weight_out.data_ptr(), freed_out.data_ptr() if F else None, F, table_in.data_ptr(),
         len_in.data_ptr(), weight_in.data_ptr(), rows, width, budget, recent)


def beam_w4_matvec_fwd(y, x, w, scales, zeros=None, group: int = 128, stream=None) -> None:
    """y [T, N] bf16 = x [T, K] bf16 times the transpose of the 4-bit weights w [N, K/2] uint8 (low
    four bits: the even column), (w - zeros) * scales per `group` columns: scales [N, K/group] bf16,
    zeros [N, K/group] uint8 in 0..15 or None (8).  The rows of x and y may be strided."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or not isinstance(w, torch.Tensor) or \
            w.dim() != 2:
        raise TypeError("x and w: expected CUDA tensors [T, K] and [N, K/2]")
    dev = x.get_device()
    T, K = x.shape
    N = w.shape[0]
    _check(x, "x", torch.bfloat16, (T, K), dev, rows=True)
    _check(y, "y", torch.bfloat16, (T, N), dev, rows=True)
    if K % 2:
        raise ValueError("x: K must be even")
    _check(w, "w", torch.uint8, (N, K // 2), dev)
    G = K // group if group > 0 else 0
    _check(scales, "scales", torch.bfloat16, (N, G), dev)
    if zeros is not None:
        _check(zeros, "zeros", torch.uint8, (N, G), dev)
    _run("beam_w4_matvec_fwd", dev, stream, y.data_ptr(), _row_stride(y) if T else N, x.data_ptr(),
         _row_stride(x) if T else K, w.data_ptr(), scales.data_ptr(),
         None if zeros is None else zeros.data_ptr(), T, N, K, group)
