"""Plain 64-bit references of the decode operators and the error bounds of their outputs (CPU)."""
from __future__ import annotations

import math

import numpy as np
import torch

D = 128
U32 = 2.0 ** -24                      # half a step of FP32
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def cache_values(cache: torch.Tensor, scale: float) -> torch.Tensor:
    """The values a cache stands for, in 64 bits."""
    if cache.dtype == torch.uint8:
        cache = cache.view(torch.float8_e4m3fn)
        return cache.float().double() * float(np.float32(scale))
    return cache.double()


def attention(q, k_cache, v_cache, prefix, table, lens, q_len, k_scale=1.0, v_scale=1.0,
              sm_scale=None, window=0, weight_in=None, fp8=False):
    """(out, lse, weights) and their error bounds, row by row over the list of keys that each sees."""
    sm = float(np.float32(D ** -0.5 if sm_scale is None else sm_scale))
    T, n_q, _ = q.shape
    n_kv = k_cache.shape[1]
    G = n_q // n_kv
    B, N = table.shape
    P = prefix.numel()
    S = k_cache.shape[0]
    out = torch.zeros((T, n_q, D), dtype=torch.float64)
    lse = torch.full((T, n_q), -math.inf, dtype=torch.float64)
    weight = torch.zeros((B, N), dtype=torch.float64) if weight_in is None else weight_in.double()
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    weight_tol = U32 * weight.abs()
    p_half = HALF[torch.float16 if fp8 else torch.bfloat16]
    for b in range(B):
        n = min(max(int(lens[b]), 0), N)
        for i in range(q_len):
            pos = n - q_len + i
            if pos < 0:
                continue
            lists = [(-1, prefix[j]) for j in range(P) if not window or P + pos - j < window]
            lists += [(j, table[b, j]) for j in range(pos + 1) if not window or pos - j < window]
            lists = [(j, int(s)) for j, s in lists if 0 <= s < S]
            if not lists:
                continue
            idx = torch.tensor([s for _, s in lists])
            js = [j for j, _ in lists]
            for h in range(n_q):
                kv = h // G
                kk = cache_values(k_cache[idx, kv], k_scale)
                vv = cache_values(v_cache[idx, kv], v_scale)
                qq = q[b * q_len + i, h].double()
                s = sm * (kk @ qq)
                # FP32 sums of 128 exact products, three roundings of the scaled score, exp2's own
                ds = float((abs(sm) * (kk.abs() @ qq.abs())).max()) * 128 * U32 * 2 + \
                    float(s.abs().max()) * 8 * U32
                z = torch.logsumexp(s, 0)
                pr = torch.exp(s - z)
                t = b * q_len + i
                out[t, h] = pr @ vv
                lse[t, h] = z
                rel = 2 * ds + 2.0 ** -20 + (len(js) + 64) * U32
                out_tol[t, h] = HALF[torch.bfloat16] * out[t, h].abs() + \
                    (p_half + rel) * (pr @ vv.abs())
                lse_tol[t, h] = ds + (len(js) + 64) * U32 + 4 * U32 * abs(float(z))
                for j, p in zip(js, pr.tolist()):
                    if j >= 0:
                        weight[b, j] += p
                        weight_tol[b, j] += (rel + 2 * U32 * n_q * q_len) * p + 2.0 ** -120
    weight_tol += 2 * U32 * weight.abs()
    return (out, lse, weight), (out_tol, lse_tol, weight_tol)


def evict(table, lens, weight, budget, recent, freed_width):
    """Exact result of the eviction, entry by entry (numpy)."""
    rows, width = table.shape
    t_out = np.full((rows, width), -1, np.int64)
    w_out = np.zeros((rows, width), np.float32)
    freed = np.full((rows, freed_width), -1, np.int64)
    n_out = np.zeros(rows, np.int32)
    for r in range(rows):
        n = min(max(int(lens[r]), 0), width)
        stay = list(range(n))
        if n > budget:
            old = n - recent
            order = sorted(range(old), key=lambda j: (
                1 if np.isnan(weight[r, j]) else 0,
                -float(weight[r, j]) if not np.isnan(weight[r, j]) else 0.0, j))
            stay = sorted(order[:budget - recent]) + list(range(old, n))
        left = sorted(set(range(n)) - set(stay))
        n_out[r] = len(stay)
        t_out[r, :len(stay)] = table[r, stay]
        w_out[r, :len(stay)] = weight[r, stay]
        freed[r, :len(left)] = table[r, left]
    return t_out, n_out, w_out, freed


def w4_matvec(x, w, scales, zeros, group):
    """(y, error bound) in 64 bits."""
    N, half = w.shape
    q = torch.empty((N, 2 * half), dtype=torch.float64)
    q[:, 0::2] = (w % 16).double()
    q[:, 1::2] = (w // 16).double()
    z = 8.0 if zeros is None else zeros.double().repeat_interleave(group, 1)
    q = (q - z) * scales.double().repeat_interleave(group, 1)
    xd = x.double()
    y = xd @ q.t()
    K = 2 * half
    chain = K // 16 + 2 * (K // group) + 16
    return y, HALF[torch.bfloat16] * y.abs() + chain * 2 * U32 * (xd.abs() @ q.abs().t())
