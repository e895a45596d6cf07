"""Decode steps of one Beam attention sublayer (a full-attention, NoPE layer) on a bounded cache.

A batch of samples shares one prompt.  Each step runs the sublayer as a server would, every step in
the library's kernels:

    x -> 4-bit QKV + gate projection -> Q/K norm + SSMax, K and V into the cache
      -> attention over the shared prompt and each sample's own tokens, gathering key weights
      -> sigmoid gate -> 4-bit output projection -> boundary (residual stream, next sublayer's x)

and evicts, once a sample's own tokens pass the budget plus some slack, those with the least
accumulated attention weight; their slots go back to the free list.

    python examples/decode_sublayer.py --batch 64 --prompt 8192 --steps 200
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import residual_stream_norm_gb300 as rsn

D = rsn.HEAD_DIM


class W4Linear:
    """A [K, N] projection held in 4 bits: the nearest of 16 levels per group of input columns."""

    def __init__(self, weight: torch.Tensor, group: int = 128):
        N, K = weight.shape
        g = weight.float().view(N, K // group, group)
        lo, hi = g.amin(2), g.amax(2)
        self.group = group
        self.scales = ((hi - lo) / 15).clamp(min=1e-8).bfloat16()
        s = self.scales.float()
        self.zeros = (-lo / s).round().clamp(0, 15).to(torch.uint8)
        q = (g / s[:, :, None] + self.zeros[:, :, None]).round().clamp(0, 15).to(torch.uint8)
        q = q.view(N, K)
        self.w = q[:, 0::2] | q[:, 1::2] << 4

    def __call__(self, y: torch.Tensor, x: torch.Tensor) -> torch.Tensor:
        rsn.beam_w4_matvec_fwd(y, x, self.w, self.scales, self.zeros, group=self.group)
        return y


class DecodeSublayer:
    def __init__(self, batch: int, prompt_len: int, budget: int, slack: int, recent: int,
                 hidden: int = 5120, n_q: int = 48, n_kv: int = 8, residual_index: int = 12,
                 cache_dtype: int = rsn.CACHE_FP8_E4M3, seed: int = 0):
        self.n_q, self.n_kv, self.n = n_q, n_kv, residual_index
        self.budget, self.recent, self.width = budget, recent, budget + slack
        self.cache_dtype = cache_dtype
        self.k_scale, self.v_scale = (0.05, 0.05) if cache_dtype else (1.0, 1.0)
        g = torch.Generator(device="cuda").manual_seed(seed)

        def randn(*shape, std=1.0):
            return torch.randn(shape, generator=g, device="cuda") * std

        def bf16(*shape, **kw):
            return torch.empty(shape, device="cuda", dtype=torch.bfloat16, **kw)

        std = hidden ** -0.5
        rows = (n_q + 2 * n_kv + n_q) * D                        # Q, K, V, gate
        self.qkvg_proj = W4Linear(randn(rows, hidden, std=std))
        self.o_proj = W4Linear(randn(hidden, n_q * D, std=(n_q * D) ** -0.5))
        self.wq, self.wk = ((1 + 0.1 * randn(D)).bfloat16() for _ in range(2))
        self.gate_bias = randn(n_q)
        self.w_post, self.w_pre = ((1 + 0.1 * randn(hidden)).bfloat16() for _ in range(2))

        # the prompt, as a prefill left it in the cache, and a free list of the other slots
        num_slots = prompt_len + batch * self.width
        kind = torch.uint8 if cache_dtype else torch.bfloat16
        self.k_cache = torch.zeros((num_slots, n_kv, D), device="cuda", dtype=kind)
        self.v_cache = torch.zeros_like(self.k_cache)
        for cache, scale in ((self.k_cache, self.k_scale), (self.v_cache, self.v_scale)):
            for i in range(0, prompt_len, 8192):
                x = randn(min(8192, prompt_len - i), n_kv, D)
                if cache_dtype:
                    x = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                cache[i:i + x.shape[0]] = x
        self.prompt = torch.arange(prompt_len, device="cuda")
        self.free = list(range(num_slots - 1, prompt_len - 1, -1))
        self.pos = torch.full((batch,), prompt_len, dtype=torch.int64, device="cuda")

        self.table = torch.full((batch, self.width), -1, dtype=torch.int64, device="cuda")
        self.len = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.weight = torch.zeros((batch, self.width), device="cuda")
        self.freed = torch.empty((batch, max(1, slack)), dtype=torch.int64, device="cuda")
        self.own = 0                                             # tokens of each sample in the cache
        self.workspace = torch.empty(rsn.beam_attn_prefix_workspace(
            batch, 1, n_q, n_kv, prompt_len, self.width, key_weights=True), dtype=torch.uint8,
            device="cuda")
        self.qkvg = bf16(batch, rows)
        self.attn, self.gated = bf16(batch, n_q, D), bf16(batch, n_q * D)
        self.out = bf16(batch, hidden)
        self.h, self.x = randn(batch, hidden).bfloat16(), randn(batch, hidden).bfloat16()

    def step(self) -> torch.Tensor:
        """One token of each sample: updates h and x in place and returns the attention's output."""
        B, nq, nk = self.x.shape[0], self.n_q, self.n_kv
        if self.own == self.width:
            self.evict()
        slots = torch.tensor([self.free.pop() for _ in range(B)], device="cuda")
        self.table[:, self.own] = slots
        self.own += 1
        self.len.fill_(self.own)

        self.qkvg_proj(self.qkvg, self.x)
        q, k, v, gate = self.qkvg.split([nq * D, nk * D, nk * D, nq * D], dim=1)
        q, k, v = (t.unflatten(1, (-1, D)) for t in (q, k, v))
        rsn.beam_qk_norm_ssmax_kv_fwd(q, k, v, self.wq, self.wk, self.pos, slots, self.k_cache,
                                      self.v_cache, cache_dtype=self.cache_dtype,
                                      k_scale=self.k_scale, v_scale=self.v_scale)
        rsn.beam_attn_prefix_fwd(self.attn, q, self.k_cache, self.v_cache, self.prompt, self.table,
                                 self.len, self.workspace, cache_dtype=self.cache_dtype,
                                 k_scale=self.k_scale, v_scale=self.v_scale,
                                 key_weight_in=self.weight, key_weight_out=self.weight)
        rsn.beam_attn_gate_fwd(self.gated, self.attn.view(B, nq * D), gate, self.gate_bias, nq)
        self.o_proj(self.out, self.gated)
        rsn.beam_boundary_fwd(self.h, self.x, self.h, self.out, self.w_post, self.w_pre, self.n)
        self.pos += 1
        return self.attn

    def evict(self) -> None:
        """Bring every sample back to the budget; the slots that leave are free again."""
        rsn.beam_kv_evict_fwd(self.table, self.len, self.weight, self.freed, self.table, self.len,
                              self.weight, self.budget, self.recent)
        self.own = self.budget
        self.free += self.freed[self.freed >= 0].tolist()


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=64)
    ap.add_argument("--prompt", type=int, default=8192)
    ap.add_argument("--budget", type=int, default=96)
    ap.add_argument("--slack", type=int, default=32)
    ap.add_argument("--recent", type=int, default=32)
    ap.add_argument("--steps", type=int, default=200)
    args = ap.parse_args()
    rsn.build()
    layer = DecodeSublayer(args.batch, args.prompt, args.budget, args.slack, args.recent)
    for _ in range(3):
        layer.step()
    torch.cuda.synchronize()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    for _ in range(args.steps):
        layer.step()
    b.record()
    torch.cuda.synchronize()
    us = a.elapsed_time(b) / args.steps * 1e3
    print(f"{args.steps} steps of {args.batch} samples behind a prompt of {args.prompt}: {us:.1f} us "
          f"a step, {layer.own} own tokens kept, {len(layer.free)} slots free, rms of h "
          f"{layer.h.float().square().mean().sqrt().item():.3f}")


if __name__ == "__main__":
    main()
