"""Plain 64-bit references of the operators of a draft-checking decode step and the error bounds of their
outputs (CPU).  Bounds count half a step of each rounded type (BF16 2^-8, FP16 2^-11, FP32 2^-24 relative),
two of FP32 for each addition inside a matrix instruction, which may cut where FP32 rounds."""
from __future__ import annotations

import math

import numpy as np
import torch

import oracle

D = 128
U32 = 2.0 ** -24
BF16, FP16 = 2.0 ** -8, 2.0 ** -11
UNIT = 1 << 44


def kv4_write(x, group):
    """(codes [T, n, 64] uint8, scales [T, n, 128 / group, 2] bf16) of rows x [T, n, 128] bf16."""
    T, n, _ = x.shape
    v = x.float().view(T, n, D // group, group).numpy()
    codes = np.zeros((T, n, D // group, group), np.uint8)
    scales = torch.zeros((T, n, D // group, 2), dtype=torch.bfloat16)
    for i in np.ndindex(T, n, D // group):
        with np.errstate(over="ignore", invalid="ignore"):
            lo, hi = v[i].min(), v[i].max()
            span = np.float32(hi - lo)
        if not np.isfinite(v[i]).all() or not np.isfinite(span):
            scales[i + (0,)] = float("nan")
            continue
        scale = torch.tensor(span / np.float32(15)).bfloat16()
        scales[i + (0,)], scales[i + (1,)] = scale, float(lo)
        if float(scale) > 0:
            codes[i] = np.minimum(np.rint((v[i] - lo) / np.float32(float(scale))), 15)
    c = codes.reshape(T, n, D)
    return torch.from_numpy(c[:, :, 0::2] | c[:, :, 1::2] << 4), scales


def kv4_values(codes, scales):
    """[..., 128] in 64 bits; also scale * code and |minimum| of each place."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).double()
    per = D // scales.shape[-2]
    s = scales[..., 0].double().repeat_interleave(per, -1)
    m = scales[..., 1].double().repeat_interleave(per, -1)
    return m + s * c, s * c, m.abs()


def kv4_attention(q, k_cache, v_cache, k_scales, v_scales, table, lens, q_len, sm_scale=None, window=0,
                  n_sink=0):
    """((out, lse), (their bounds)), row by row over the list of keys that each sees."""
    sm = float(np.float32(D ** -0.5 if sm_scale is None else sm_scale))
    T, n_q, _ = q.shape
    S, n_kv, _ = k_cache.shape
    G = n_q // n_kv
    B, N = table.shape
    out = torch.zeros((T, n_q, D), dtype=torch.float64)
    lse = torch.full((T, n_q), -math.inf, dtype=torch.float64)
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(B):
        n = min(max(int(lens[b]), 0), N)
        for i in range(q_len):
            p = n - q_len + i
            if p < 0:
                continue
            js = [j for j in range(p + 1) if not window or p - j < window or j < n_sink]
            at = table[b, js]
            at = at[(at >= 0) & (at < S)]
            if not at.numel():
                continue
            t = b * q_len + i
            for kv in range(n_kv):
                kk, ksc, kmin = kv4_values(k_cache[at, kv], k_scales[at, kv])
                vv, vsc, vmin = kv4_values(v_cache[at, kv], v_scales[at, kv])
                hs = slice(kv * G, kv * G + G)
                qq = q[t, hs].double()
                s = sm * qq @ kk.t()
                # 128 exact products in FP32 by groups, then scaled; sum q in FP32; exp2's argument
                size = abs(sm) * qq.abs() @ (ksc + kmin).t()
                ds = size.amax(1) * (2 * 128 + 32) * U32 + 8 * U32 * s.abs().amax(1)
                z = torch.logsumexp(s, 1)
                w = torch.exp(s - z[:, None])
                rel = (2 * ds + 2.0 ** -20 + 2 * (at.numel() + 64) * U32)[:, None]
                out[t, hs] = w @ vv
                lse[t, hs] = z
                out_tol[t, hs] = BF16 * out[t, hs].abs() + (FP16 + rel) * (w @ vsc) + rel * (w @ vmin) + \
                    15 * 2.0 ** -32 * float(v_scales[at, kv, :, 0].double().max()) * at.numel()
                lse_tol[t, hs] = ds + 2.0 ** -20 + 2 * (at.numel() + 64) * U32 + 4 * U32 * z.abs()
    return (out, lse), (out_tol, lse_tol)


def moe_route(x, router_w, router_bias):
    """(ids, weights) as the framework's grouped top-k gives them on logits rounded once to FP32."""
    z = (x.double() @ router_w.double().t()).float()
    return oracle.grouped_topk(z.numpy(), router_bias.numpy())


def moe_layer(x, ids, weights, w13, w2, first, scaling):
    """(out, bound): x [T, H], ids and weights [T, 8], w13(e) [2F, H] and w2(e) [H, F] by local expert."""
    T, H = x.shape
    out = torch.zeros((T, H), dtype=torch.float64)
    tol = torch.zeros_like(out)
    total = torch.zeros_like(out)
    for t in range(T):
        for k in range(8):
            e = int(ids[t, k]) - first
            if w13(e) is None:
                continue
            a13, a2, xt = w13(e).double(), w2(e).double(), x[t].double()
            F = a2.shape[1]
            gu = a13 @ xt
            # FP32 sums in steps of 16 products, over 8 warps: at most H / 128 + 8 + 16 additions
            d = (H / 128 + 24) * 2 * U32 * (a13.abs() @ xt.abs())
            g, u = gu[:F], gu[F:]
            sig = torch.sigmoid(g)
            a = g * sig * u
            # |silu'| <= 1.1; then two BF16 parts
            da = 1.1 * d[:F] * u.abs() + (g * sig).abs() * d[F:] + (BF16 ** 2 + 16 * U32) * a.abs()
            da += 1.1 * d[:F] * d[F:]
            c = float(np.float32(scaling)) * float(weights[t, k])
            y = a2 @ a
            out[t] += c * y
            size = a2.abs() @ a.abs()
            total[t] += abs(c) * size
            tol[t] += abs(c) * (a2.abs() @ da * (1 + 2.0 ** -7) + (F / 128 + 32) * 2 * U32 * size)
    tol += 16 * U32 * total + BF16 * (out.abs() + tol)
    return out, tol


def verify(tokens, target, draft, u_accept, u_sample, lens=None):
    """(tokens_out, accepted), in whole numbers."""
    B, k = tokens.shape
    V = target.shape[2]
    f = lambda p: np.nan_to_num(np.clip(p.double().numpy(), 0.0, 1.0), nan=0.0)  # noqa: E731
    units = lambda p: [int(x) for x in np.rint(f(p) * UNIT).tolist()]  # noqa: E731
    out = np.full((B, k + 1), -1, np.int64)
    acc = np.zeros(B, np.int32)
    for b in range(B):
        n = k if lens is None else min(max(int(lens[b]), 0), k)
        a = 0
        while a < n:
            x = int(tokens[b, a])
            if not 0 <= x < V:
                break
            q = 1.0 if draft is None else float(draft[b, a, x])
            if not float(u_accept[b, a]) * q < float(target[b, a, x]):
                break
            a += 1
        w = p = units(target[b, a])
        if a < n:
            if draft is not None:
                w = [max(i - j, 0) for i, j in zip(p, units(draft[b, a]))]
            else:
                x = int(tokens[b, a])
                w = [0 if v == x else i for v, i in enumerate(p)]
            if not any(w):
                w = p
        S, run, token = sum(w), 0, -1
        u = float(u_sample[b])
        u = 0.0 if u != u else min(max(u, 0.0), float(np.float32(0.99999994)))
        border = int(u * 2.0 ** 24) * S >> 24
        for v, i in enumerate(w):
            run += i
            if run > border:
                token = v
                break
        out[b, :a] = tokens[b, :a]
        out[b, a] = token
        acc[b] = a
    return out, acc
