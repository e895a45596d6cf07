"""Decoding with drafted tokens on one Beam layer: every sequence drafts a few tokens, one step of the layer
runs all of them at once, and the verification keeps what the target agrees with.

The step, as a server would run it (a sliding-window, RoPE layer with the first tokens in sight):

    x -> 4-bit QKV + gate projection -> Q/K norm + RoPE -> K and V into the 4-bit cache
      -> attention over each sequence's window and first tokens -> sigmoid gate -> 4-bit output projection
      -> boundary -> mixture-of-experts layer -> boundary -> probabilities -> verification

A sequence's tokens behind the last accepted one are forgotten by its length alone: the next step writes over
them.  The drafter is a table of what follows a token.

    python examples/draft_step.py --batch 16 --drafts 3 --steps 100
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import residual_stream_norm_gb300 as rsn
from examples.decode_sublayer import W4Linear

D = rsn.HEAD_DIM


class DraftDecoder:
    def __init__(self, batch: int, drafts: int, max_len: int, hidden: int = 5120, n_q: int = 48, n_kv: int = 8,
                 expert_width: int = 320, vocab: int = 4096, window: int = 512, n_sink: int = 4,
                 group: int = 64, residual_index: int = 12, seed: int = 0):
        self.k, self.n_q, self.n_kv, self.n = drafts, n_q, n_kv, residual_index
        self.window, self.n_sink, self.group, self.max_len = window, n_sink, group, max_len
        self.gen = g = torch.Generator(device="cuda").manual_seed(seed)

        def randn(*shape, std=1.0):
            return torch.randn(shape, generator=g, device="cuda") * std

        def bf16(*shape):
            return torch.empty(shape, device="cuda", dtype=torch.bfloat16)

        std, T = hidden ** -0.5, batch * (drafts + 1)
        rows = (2 * n_q + 2 * n_kv) * D                          # Q, K, V, gate
        self.qkvg_proj = W4Linear(randn(rows, hidden, std=std))
        self.o_proj = W4Linear(randn(hidden, n_q * D, std=(n_q * D) ** -0.5))
        self.wq, self.wk = ((1 + 0.1 * randn(D)).bfloat16() for _ in range(2))
        self.gate_bias = randn(n_q)
        self.norms = [(1 + 0.1 * randn(hidden)).bfloat16() for _ in range(4)]
        self.router, self.router_bias = randn(256, hidden, std=std), randn(256, std=0.05)
        self.w_gate_up = randn(256, 2 * expert_width, hidden, std=std).bfloat16()
        self.w_down = randn(256, hidden, expert_width, std=expert_width ** -0.5).bfloat16()
        self.embedding, self.head = randn(vocab, hidden).bfloat16(), randn(vocab, hidden, std=3 * std).bfloat16()
        self.draft_table = torch.softmax(randn(vocab, vocab, std=2.0), 1)

        # each sequence has its places in the cache, in pages of 16 at random
        pages = torch.randperm(batch * -(-max_len // 16), generator=g, device="cuda").view(batch, -1)
        self.table = (pages[:, :, None] * 16 + torch.arange(16, device="cuda")).flatten(1)[:, :max_len].contiguous()
        slots = int(self.table.max()) + 1
        self.k_cache, self.v_cache = (torch.zeros((slots, n_kv, D // 2), device="cuda", dtype=torch.uint8)
                                      for _ in range(2))
        self.k_scales, self.v_scales = (torch.zeros((slots, n_kv, D // group, 2), device="cuda",
                                                    dtype=torch.bfloat16) for _ in range(2))
        self.len = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.last = torch.randint(0, vocab, (batch,), generator=g, device="cuda")

        self.attn_workspace = torch.empty(rsn.beam_attn_kv4_workspace(
            batch, drafts + 1, n_q, n_kv, max_len, window, n_sink), dtype=torch.uint8, device="cuda")
        self.moe_workspace = torch.empty(rsn.beam_moe_layer_workspace(T, hidden, expert_width),
                                         dtype=torch.uint8, device="cuda")
        self.qkvg, self.attn, self.gated = bf16(T, rows), bf16(T, n_q, D), bf16(T, n_q * D)
        self.out, self.moe = bf16(T, hidden), bf16(T, hidden)
        self.y, self.x = bf16(T, hidden), bf16(T, hidden)
        self.ids = torch.empty((T, 8), dtype=torch.int32, device="cuda")
        self.weights = torch.empty((T, 8), device="cuda")
        self.tokens = torch.empty((batch, drafts + 1), dtype=torch.int64, device="cuda")
        self.accepted = torch.empty(batch, dtype=torch.int32, device="cuda")

    def draft(self):
        """k tokens of each sequence and the distributions that they were drawn from."""
        B, V = self.len.shape[0], self.draft_table.shape[0]
        tokens = torch.empty((B, self.k), dtype=torch.int64, device="cuda")
        probs = torch.empty((B, self.k, V), device="cuda")
        token = self.last
        for i in range(self.k):
            probs[:, i] = self.draft_table[token]
            token = tokens[:, i] = torch.multinomial(probs[:, i], 1, generator=self.gen)[:, 0]
        return tokens, probs

    def step(self) -> torch.Tensor:
        """One step: returns the tokens that each sequence gained, -1 behind them."""
        B, L, nq, nk = self.len.shape[0], self.k + 1, self.n_q, self.n_kv
        drafted, draft_probs = self.draft()
        tokens = torch.cat((self.last[:, None], drafted), 1)
        h = self.embedding[tokens.flatten()]
        x = (h.float() * h.float().square().mean(1, keepdim=True).rsqrt()).bfloat16()
        pos = self.len.long()[:, None] + torch.arange(L, device="cuda")
        slots = self.table.gather(1, pos).flatten()
        self.seq_len = self.len + L

        self.qkvg_proj(self.qkvg, x)
        q, k, v, gate = self.qkvg.split([nq * D, nk * D, nk * D, nq * D], dim=1)
        q, k, v = (t.unflatten(1, (-1, D)) for t in (q, k, v))
        rsn.beam_qk_norm_rope_fwd(q, k, self.wq, self.wk, pos.flatten())
        rsn.beam_kv4_write_fwd(self.k_cache, self.v_cache, self.k_scales, self.v_scales, k, v, slots,
                               group=self.group)
        rsn.beam_attn_kv4_fwd(self.attn, q, self.k_cache, self.v_cache, self.k_scales, self.v_scales, self.table,
                              self.seq_len, self.attn_workspace, group=self.group, window=self.window,
                              n_sink=self.n_sink)
        rsn.beam_attn_gate_fwd(self.gated, self.attn.flatten(1), gate, self.gate_bias, nq)
        self.o_proj(self.out, self.gated)
        rsn.beam_boundary_fwd(h, self.y, h, self.out, *self.norms[:2], self.n)
        rsn.beam_moe_layer_fwd(self.moe, self.y, self.router, self.router_bias, self.w_gate_up, self.w_down,
                               self.moe_workspace, topk_ids_out=self.ids, topk_w_out=self.weights)
        rsn.beam_boundary_fwd(h, self.x, h, self.moe, *self.norms[2:], self.n + 1)

        self.probs = torch.softmax((self.x @ self.head.t()).float(), 1).view(B, L, -1)
        u = torch.rand((B, L), generator=self.gen, device="cuda")
        self.drawn = drafted, draft_probs, u
        rsn.beam_draft_verify_fwd(self.tokens, self.accepted, drafted, self.probs, draft_probs,
                                  u[:, :self.k].contiguous(), u[:, self.k].contiguous())
        # the cache keeps the last token and the accepted ones; the drawn one comes next
        self.len += 1 + self.accepted
        self.last = self.tokens.gather(1, self.accepted.long()[:, None])[:, 0]
        return self.tokens


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=16)
    ap.add_argument("--drafts", type=int, default=3)
    ap.add_argument("--steps", type=int, default=100)
    args = ap.parse_args()
    rsn.build()
    m = DraftDecoder(args.batch, args.drafts, (args.steps + 3) * (args.drafts + 1) + 16)
    for _ in range(3):
        m.step()
    torch.cuda.synchronize()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    before = int(m.len.sum())
    a.record()
    for _ in range(args.steps):
        m.step()
    b.record()
    torch.cuda.synchronize()
    n = int(m.len.sum()) - before
    print(f"{args.steps} steps of {args.batch} sequences with {args.drafts} drafts: "
          f"{a.elapsed_time(b) / args.steps * 1e3:.1f} us a step, {n / args.steps / args.batch:.2f} tokens a step "
          f"and sequence")


if __name__ == "__main__":
    main()
