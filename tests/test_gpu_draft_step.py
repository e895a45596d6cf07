"""The operators of a draft-checking step together, as a server uses them (examples/draft_step.py): each step's
results compared with plain 64-bit and whole-number computations on the same state (needs a GB300)."""
import importlib.util
import os
import sys

import pytest
import torch

import residual_stream_norm_gb300 as rsn
from tests import _draft_ref as ref
from tests._gpu import lib

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    if ROOT not in sys.path:
        sys.path.insert(0, ROOT)
    spec = importlib.util.spec_from_file_location("draft_step", os.path.join(ROOT, "examples", "draft_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("drafts,window", [(0, 0), (3, 9), (4, 0)])
def test_steps(drafts, window):
    lib()
    B, n_q, n_kv, H = 3, 12, 2, 256
    s = example().DraftDecoder(B, drafts, 80, hidden=H, n_q=n_q, n_kv=n_kv, expert_width=40, vocab=300,
                               window=window, n_sink=2, group=32)
    w13, w2 = s.w_gate_up.cpu(), s.w_down.cpu()
    gained = 0
    for _ in range(10):
        before = s.len.cpu()
        tokens = s.step().cpu()
        torch.cuda.synchronize()
        L = drafts + 1
        # what this step wrote into the cache are its own K and V
        pos = before.long()[:, None] + torch.arange(L)
        slots = s.table.cpu().gather(1, pos).flatten()
        kv = s.qkvg.cpu()[:, n_q * 128:(n_q + 2 * n_kv) * 128].view(-1, 2, n_kv, 128)
        for i, x in enumerate(("k", "v")):
            codes, scales = ref.kv4_write(kv[:, i], 32)
            assert torch.equal(getattr(s, x + "_cache").cpu()[slots], codes)
            assert torch.equal(getattr(s, x + "_scales").cpu()[slots], scales)
        # attention over what the cache holds now
        q = s.qkvg[:, :n_q * 128].cpu().view(-1, n_q, 128)
        (want, _), (tol, _) = ref.kv4_attention(q, s.k_cache.cpu(), s.v_cache.cpu(), s.k_scales.cpu(),
                                                s.v_scales.cpu(), s.table.cpu(), s.seq_len.cpu(), L,
                                                window=window, n_sink=2)
        assert bool(((s.attn.cpu().double() - want).abs() <= tol).all())
        # the layer of experts
        ids, weights = ref.moe_route(s.y.cpu(), s.router.cpu(), s.router_bias.cpu())
        assert (s.ids.cpu().numpy() == ids).all() and (s.weights.cpu().numpy() == weights).all()
        want, tol = ref.moe_layer(s.y.cpu(), ids, weights, lambda e: w13[e], lambda e: w2[e], 0, 2.5)
        assert bool(((s.moe.cpu().double() - want).abs() <= tol).all())
        # the tokens
        drafted, draft_probs, u = (t.cpu() for t in s.drawn)
        out, acc = ref.verify(drafted, s.probs.cpu(), draft_probs, u[:, :drafts], u[:, drafts])
        assert (tokens.numpy() == out).all() and (s.accepted.cpu().numpy() == acc).all()
        assert torch.equal(s.len.cpu(), before + 1 + s.accepted.cpu())
        gained += int(s.accepted.sum())
    assert rsn.beam_device_faults() == 0
    if drafts:
        assert gained > 0
