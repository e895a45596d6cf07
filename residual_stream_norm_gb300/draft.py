"""Python binding of the operators of a decode step that checks drafted tokens (``include/beam_draft.h``):
the KV cache held in 4 bits (its write and its attention), a whole mixture-of-experts layer for a few
tokens, and the verification of drafted tokens.

The functions carry the C names, check and marshal their arguments, and raise ``BeamError`` on a non-zero
status; they are reached as ``residual_stream_norm_gb300.beam_...``.
"""
from __future__ import annotations

import ctypes

import torch

from .decode import _SM_SCALE, HEAD_DIM, _bf16, _check, _f32, _head_rows, _i32, _i64, _run, _u8

EXPERTS, TOP_K = 256, 8


def declare(so: ctypes.CDLL) -> None:
    """Argument types of the entry points of ``beam_draft.h``."""
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    so.beam_kv4_write_fwd.argtypes = [vp, vp, vp, vp, i64, i32, vp, i64, vp, i64, vp, i64, i32, i32, vp]
    so.beam_kv4_write_fwd.restype = ctypes.c_int
    so.beam_attn_kv4_workspace.argtypes = [i32, i32, i32, i32, i64, i64, i64]
    so.beam_attn_kv4_workspace.restype = i64
    so.beam_attn_kv4_fwd.argtypes = [vp, i64, vp, vp, i64, vp, vp, vp, vp, i64, i32, vp, i64, i64, vp, i32,
                                     i32, i32, i32, i32, f32, i64, i64, vp, i64, vp]
    so.beam_attn_kv4_fwd.restype = ctypes.c_int
    so.beam_moe_layer_workspace.argtypes = [i64, i32, i32, i32]
    so.beam_moe_layer_workspace.restype = i64
    so.beam_moe_layer_fwd.argtypes = [vp, i64, vp, vp, vp, i64, vp, vp, vp, vp, i32, i32, f32, i64, i32,
                                      i32, vp, i64, vp]
    so.beam_moe_layer_fwd.restype = ctypes.c_int
    so.beam_draft_verify_fwd.argtypes = [vp, vp, vp, vp, vp, i64, i64, vp, i64, i64, i32, vp, vp, i64, i32,
                                         i64, vp]
    so.beam_draft_verify_fwd.restype = ctypes.c_int


def _int(x, bits: int = 32):
    """x, or -1, which every size here refuses, where the C type cannot hold it (ctypes would cut it off)."""
    return x if -1 << bits - 1 <= x < 1 << bits - 1 else -1


# As in decode.py: good arguments cost one expression; only when it fails do the checks find out what to say.

def _cache_good(k_cache, v_cache, k_scales, v_scales, dev, groups):
    S, n_kv, half = k_cache.shape
    shape = (S, n_kv, groups, 2)
    return (half == HEAD_DIM // 2 and k_cache.dtype is _u8 and v_cache.dtype is _u8 and
            v_cache.shape == k_cache.shape and k_scales.dtype is _bf16 and v_scales.dtype is _bf16 and
            k_scales.shape == shape and v_scales.shape == shape and
            k_cache.get_device() == dev and v_cache.get_device() == dev and
            k_scales.get_device() == dev and v_scales.get_device() == dev and
            k_cache.is_contiguous() and v_cache.is_contiguous() and
            k_scales.is_contiguous() and v_scales.is_contiguous())


def _cache_check(k_cache, v_cache, k_scales, v_scales, dev, groups) -> None:
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 3:
        raise TypeError(f"k_cache: expected a CUDA uint8 tensor [num_slots, n_kv, {HEAD_DIM // 2}]")
    S, n_kv = k_cache.shape[:2]
    for t, nm in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _check(t, nm, _u8, (S, n_kv, HEAD_DIM // 2), dev)
    for t, nm in ((k_scales, "k_scales"), (v_scales, "v_scales")):
        _check(t, nm, _bf16, (S, n_kv, groups, 2), dev)


def _groups(group: int) -> int:
    return HEAD_DIM // group if group > 0 else 0


def beam_kv4_write_fwd(k_cache, v_cache, k_scales, v_scales, k, v, slot_mapping, group: int = 128,
                       stream=None) -> None:
    """Write k, v [T, n_kv, 128] bf16 (row-strided views allowed) into the slots slot_mapping [T] int64 of a
    cache held in 4 bits: k_cache, v_cache [num_slots, n_kv, 64] uint8 (low four bits: the even column),
    k_scales, v_scales [num_slots, n_kv, 128 / group, 2] bf16 (scale, minimum); a code stands for
    minimum + scale * code.  Negative or out-of-range slots are skipped."""
    T, n_kv, k_stride, dev = _head_rows(k, "k")
    Tv, nv, v_stride, vdev = _head_rows(v, "v")
    if (Tv, nv, vdev) != (T, n_kv, dev):
        raise ValueError("v must have k's shape and device")
    groups = _groups(group)
    try:
        good = (_cache_good(k_cache, v_cache, k_scales, v_scales, dev, groups) and
                k_cache.shape[1] == n_kv and slot_mapping.dtype is _i64 and
                slot_mapping.shape == (T,) and slot_mapping.get_device() == dev and
                slot_mapping.is_contiguous())
    except (AttributeError, ValueError):
        good = False
    if not good:
        _cache_check(k_cache, v_cache, k_scales, v_scales, dev, groups)
        _check(slot_mapping, "slot_mapping", _i64, (T,), dev)
        raise ValueError(f"k has {n_kv} heads, the cache {k_cache.shape[1]}")
    _run("beam_kv4_write_fwd", dev, stream, k_cache.data_ptr(), v_cache.data_ptr(), k_scales.data_ptr(),
         v_scales.data_ptr(), k_cache.shape[0], group, k.data_ptr(), k_stride, v.data_ptr(), v_stride,
         slot_mapping.data_ptr(), T, n_kv, HEAD_DIM)


def beam_attn_kv4_workspace(B: int, q_len: int, n_q_heads: int, n_kv_heads: int, table_width: int,
                            window: int = 0, n_sink: int = 0) -> int:
    """Bytes of workspace ``beam_attn_kv4_fwd`` needs for these sizes (host only)."""
    from . import BeamError, lib
    n = lib().beam_attn_kv4_workspace(_int(B), _int(q_len), _int(n_q_heads), _int(n_kv_heads), _int(table_width, 64),
                                      _int(window, 64), _int(n_sink, 64))
    if n < 0:
        raise BeamError("beam_attn_kv4_workspace", n)
    return n


def beam_attn_kv4_fwd(out, q, k_cache, v_cache, k_scales, v_scales, slot_table, seq_len, workspace,
                      group: int = 128, sm_scale: float | None = None, window: int = 0, n_sink: int = 0,
                      lse_out=None, stream=None) -> None:
    """Attention of a decode batch over a cache held in 4 bits (the layout of ``beam_kv4_write_fwd``).

    out, q: [B*q_len, n_q, 128] bf16 (row-strided views allowed); slot_table [B, N] int64 (rows may be
    strided); seq_len [B] int32; workspace: a contiguous uint8 tensor of at least
    ``beam_attn_kv4_workspace`` bytes; lse_out [B*q_len, n_q] fp32.  The last q_len entries of a sequence
    are its query tokens.  With a window, the first n_sink keys stay visible.  sm_scale defaults to
    1/sqrt(128)."""
    T, nq, q_stride, dev = _head_rows(q, "q")
    oT, oq, out_stride, odev = _head_rows(out, "out")
    if oT != T or oq != nq or odev != dev:
        raise ValueError("out must have q's shape and device")
    groups = _groups(group)
    try:
        B, N = slot_table.shape
        good = (_cache_good(k_cache, v_cache, k_scales, v_scales, dev, groups) and
                slot_table.dtype is _i64 and slot_table.get_device() == dev and
                (slot_table.is_contiguous() or slot_table.stride(1) == 1) and
                seq_len.dtype is _i32 and seq_len.shape == (B,) and seq_len.get_device() == dev and
                seq_len.is_contiguous() and workspace.get_device() == dev and workspace.is_contiguous() and
                (lse_out is None or (lse_out.dtype is _f32 and lse_out.shape == (T, nq) and
                                     lse_out.get_device() == dev and lse_out.is_contiguous())))
    except (AttributeError, ValueError):
        good = False
    if not good:
        if not isinstance(slot_table, torch.Tensor) or slot_table.dim() != 2:
            raise TypeError("slot_table: expected a CUDA int64 tensor [B, N]")
        B, N = slot_table.shape
        _check(slot_table, "slot_table", _i64, (B, N), dev, rows=True)
        _check(seq_len, "seq_len", _i32, (B,), dev)
        _cache_check(k_cache, v_cache, k_scales, v_scales, dev, groups)
        if lse_out is not None:
            _check(lse_out, "lse_out", _f32, (T, nq), dev)
        raise TypeError("workspace: expected a contiguous CUDA tensor on q's device")
    if T % B if B else T:
        raise ValueError(f"q has {T} rows, not a multiple of the {B} sequences")
    S, n_kv, _ = k_cache.shape
    _run("beam_attn_kv4_fwd", dev, stream, out.data_ptr(), out_stride,
         None if lse_out is None else lse_out.data_ptr(), q.data_ptr(), q_stride, k_cache.data_ptr(),
         v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), S, group, slot_table.data_ptr(),
         slot_table.stride(0) if B > 1 else N, N, seq_len.data_ptr(), B, T // B if B else 1, nq, n_kv,
         HEAD_DIM, _SM_SCALE if sm_scale is None else sm_scale, _int(window, 64), _int(n_sink, 64),
         workspace.data_ptr(), workspace.nbytes)


def beam_moe_layer_workspace(T: int, H: int, F: int, n_local: int = EXPERTS) -> int:
    """Bytes of workspace ``beam_moe_layer_fwd`` needs for these sizes (host only)."""
    from . import BeamError, lib
    n = lib().beam_moe_layer_workspace(_int(T, 64), _int(H), _int(F), _int(n_local))
    if n < 0:
        raise BeamError("beam_moe_layer_workspace", n)
    return n


def beam_moe_layer_fwd(out, x, router_w, router_bias, w_gate_up, w_down, workspace, first_expert: int = 0,
                       routed_scaling: float = 2.5, topk_ids_out=None, topk_w_out=None,
                       stream=None) -> None:
    """A whole mixture-of-experts layer for up to 256 tokens: out [T, H] bf16 = the weighted sum of each
    token's 8 experts, out of 256, that lie in [first_expert, first_expert + n_local).

    x [T, H] bf16 (the rows of x and out may be strided); router_w [256, H], router_bias [256] fp32;
    w_gate_up [n_local, 2*F, H] (the gate's rows, then the up projection's) and w_down [n_local, H, F]
    bf16; workspace: a contiguous uint8 tensor of at least ``beam_moe_layer_workspace`` bytes;
    topk_ids_out [T, 8] int32 and topk_w_out [T, 8] fp32 or None."""
    try:
        dev = x.get_device()
        T, H = x.shape
        n_local, _, F = w_down.shape
        good = (dev >= 0 and x.dtype is _bf16 and (x.is_contiguous() or x.stride(1) == 1) and
                out.dtype is _bf16 and out.shape == (T, H) and out.get_device() == dev and
                (out.is_contiguous() or out.stride(1) == 1) and
                router_w.dtype is _f32 and router_w.shape == (EXPERTS, H) and
                router_w.get_device() == dev and router_w.is_contiguous() and
                router_bias.dtype is _f32 and router_bias.shape == (EXPERTS,) and
                router_bias.get_device() == dev and router_bias.is_contiguous() and
                w_gate_up.dtype is _bf16 and w_gate_up.shape == (n_local, 2 * F, H) and
                w_gate_up.get_device() == dev and w_gate_up.is_contiguous() and
                w_down.dtype is _bf16 and w_down.shape[1] == H and w_down.get_device() == dev and
                w_down.is_contiguous() and
                workspace.get_device() == dev and workspace.is_contiguous() and
                (topk_ids_out is None or (topk_ids_out.dtype is _i32 and
                                          topk_ids_out.shape == (T, TOP_K) and
                                          topk_ids_out.get_device() == dev and
                                          topk_ids_out.is_contiguous())) and
                (topk_w_out is None or (topk_w_out.dtype is _f32 and topk_w_out.shape == (T, TOP_K) and
                                        topk_w_out.get_device() == dev and topk_w_out.is_contiguous())))
    except (AttributeError, ValueError):
        good = False
    if not good:
        if not isinstance(x, torch.Tensor) or x.dim() != 2 or not isinstance(w_down, torch.Tensor) or \
                w_down.dim() != 3:
            raise TypeError("x and w_down: expected CUDA tensors [T, H] and [n_local, H, F]")
        dev = x.get_device()
        T, H = x.shape
        n_local, _, F = w_down.shape
        _check(x, "x", _bf16, (T, H), dev, rows=True)
        _check(out, "out", _bf16, (T, H), dev, rows=True)
        _check(router_w, "router_w", _f32, (EXPERTS, H), dev)
        _check(router_bias, "router_bias", _f32, (EXPERTS,), dev)
        _check(w_gate_up, "w_gate_up", _bf16, (n_local, 2 * F, H), dev)
        _check(w_down, "w_down", _bf16, (n_local, H, F), dev)
        if topk_ids_out is not None:
            _check(topk_ids_out, "topk_ids_out", _i32, (T, TOP_K), dev)
        if topk_w_out is not None:
            _check(topk_w_out, "topk_w_out", _f32, (T, TOP_K), dev)
        raise TypeError("workspace: expected a contiguous CUDA tensor on x's device")
    _run("beam_moe_layer_fwd", dev, stream, out.data_ptr(), out.stride(0) if T > 1 else H,
         None if topk_ids_out is None else topk_ids_out.data_ptr(),
         None if topk_w_out is None else topk_w_out.data_ptr(), x.data_ptr(),
         x.stride(0) if T > 1 else H, router_w.data_ptr(), router_bias.data_ptr(), w_gate_up.data_ptr(),
         w_down.data_ptr(), _int(first_expert), n_local, routed_scaling, T, H, F, workspace.data_ptr(),
         workspace.nbytes)


def beam_draft_verify_fwd(tokens_out, n_accepted_out, draft_tokens, target_probs, draft_probs, u_accept,
                          u_sample, draft_len=None, stream=None) -> None:
    """Verify drafted tokens: tokens_out [B, k + 1] int64 gets each sequence's accepted tokens, the one drawn
    behind them, and -1; n_accepted_out [B] int32 their number.

    draft_tokens [B, k] int64; target_probs [B, k + 1, V] fp32 or bf16; draft_probs [B, k, V] of the same
    type, or None (each drafted token was certain); u_accept [B, k], u_sample [B] fp32 in [0, 1); draft_len
    [B] int32 or None (k).  The distributions' rows are contiguous, their other strides free."""
    try:
        dev = target_probs.get_device()
        B, k1, V = target_probs.shape
        k = k1 - 1
        dt = target_probs.dtype
        good = (dev >= 0 and (dt is _f32 or dt is _bf16) and
                (target_probs.is_contiguous() or target_probs.stride(2) == 1) and
                (draft_probs is None or (draft_probs.dtype is dt and draft_probs.shape == (B, k, V) and
                                         draft_probs.get_device() == dev and
                                         (draft_probs.is_contiguous() or draft_probs.stride(2) == 1))) and
                tokens_out.dtype is _i64 and tokens_out.shape == (B, k1) and
                tokens_out.get_device() == dev and tokens_out.is_contiguous() and
                n_accepted_out.dtype is _i32 and n_accepted_out.shape == (B,) and
                n_accepted_out.get_device() == dev and n_accepted_out.is_contiguous() and
                draft_tokens.dtype is _i64 and draft_tokens.shape == (B, k) and
                draft_tokens.get_device() == dev and draft_tokens.is_contiguous() and
                u_accept.dtype is _f32 and u_accept.shape == (B, k) and u_accept.get_device() == dev and
                u_accept.is_contiguous() and
                u_sample.dtype is _f32 and u_sample.shape == (B,) and u_sample.get_device() == dev and
                u_sample.is_contiguous() and
                (draft_len is None or (draft_len.dtype is _i32 and draft_len.shape == (B,) and
                                       draft_len.get_device() == dev and draft_len.is_contiguous())))
    except (AttributeError, ValueError):
        good = False
    if not good:
        if not isinstance(target_probs, torch.Tensor) or target_probs.dim() != 3 or \
                target_probs.dtype not in (_f32, _bf16) or target_probs.shape[1] < 1:
            raise TypeError("target_probs: expected a CUDA fp32 or bf16 tensor [B, k + 1, V]")
        dev = target_probs.get_device()
        B, k1, V = target_probs.shape
        k, dt = k1 - 1, target_probs.dtype
        _check(target_probs, "target_probs", dt, (B, k1, V), dev, rows=True)
        if draft_probs is not None:
            _check(draft_probs, "draft_probs", dt, (B, k, V), dev, rows=True)
        _check(tokens_out, "tokens_out", _i64, (B, k1), dev)
        _check(n_accepted_out, "n_accepted_out", _i32, (B,), dev)
        _check(draft_tokens, "draft_tokens", _i64, (B, k), dev)
        _check(u_accept, "u_accept", _f32, (B, k), dev)
        _check(u_sample, "u_sample", _f32, (B,), dev)
        _check(draft_len, "draft_len", _i32, (B,), dev)
    ts, tp, _ = target_probs.stride()
    ds, dp = (0, 0) if draft_probs is None else draft_probs.stride()[:2]
    _run("beam_draft_verify_fwd", dev, stream, tokens_out.data_ptr(), n_accepted_out.data_ptr(),
         draft_tokens.data_ptr(), None if draft_len is None else draft_len.data_ptr(),
         target_probs.data_ptr(), ts, tp, None if draft_probs is None else draft_probs.data_ptr(), ds, dp,
         0 if dt is _f32 else 1, u_accept.data_ptr(), u_sample.data_ptr(), B, k, V)
