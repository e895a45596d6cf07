"""The decode operators together, as a server uses them: steps of an attention sublayer on a bounded
cache (examples/decode_sublayer.py), each compared with plain 64-bit computations on the same state
(needs a GB300)."""
import importlib.util
import os

import pytest
import torch

import residual_stream_norm_gb300 as rsn
from tests import _decode_ref as ref
from tests._gpu import lib

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location(
        "decode_sublayer", os.path.join(ROOT, "examples", "decode_sublayer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("cache_dtype", [rsn.CACHE_BF16, rsn.CACHE_FP8_E4M3])
def test_sublayer_steps(cache_dtype):
    lib()
    B, prompt = 3, 70
    s = example().DecodeSublayer(B, prompt, budget=6, slack=3, recent=2, hidden=256, n_q=12, n_kv=2,
                                 cache_dtype=cache_dtype)
    slots = set(range(prompt, s.k_cache.shape[0]))
    for step in range(14):
        before, x = s.weight.clone(), s.x.cpu()
        evicts = s.own == s.width
        table, weight = s.table.cpu().numpy().copy(), s.weight.cpu().numpy().copy()
        attn = s.step().cpu()
        torch.cuda.synchronize()
        assert bool(torch.isfinite(s.h).all()) and bool(torch.isfinite(s.x).all())
        if evicts:
            want = ref.evict(table, [s.width] * B, weight, s.budget, s.recent, s.width - s.budget)
            assert (s.table.cpu().numpy()[:, :s.budget] == want[0][:, :s.budget]).all()
            before = torch.from_numpy(want[2])
        # every slot is in one place
        held = s.table[:, :s.own].flatten().tolist()
        assert sorted(held + s.free) == sorted(slots)
        # the projection, and the attention over what the cache holds now
        y, tol = ref.w4_matvec(x, s.qkvg_proj.w.cpu(), s.qkvg_proj.scales.cpu(),
                               s.qkvg_proj.zeros.cpu(), s.qkvg_proj.group)
        gate = slice((s.n_q + 2 * s.n_kv) * 128, None)
        assert bool(((s.qkvg.cpu().double() - y).abs() <= tol)[:, gate].all())
        q = s.qkvg[:, :s.n_q * 128].cpu().view(B, s.n_q, 128)
        want, tol = ref.attention(q, s.k_cache.cpu(), s.v_cache.cpu(), s.prompt.cpu(),
                                  s.table.cpu(), s.len.cpu(), 1, s.k_scale, s.v_scale,
                                  weight_in=before.cpu(), fp8=cache_dtype == rsn.CACHE_FP8_E4M3)
        assert bool(((attn.double() - want[0]).abs() <= tol[0]).all())
        assert bool(((s.weight.cpu().double() - want[2]).abs() <= tol[2]).all())
    assert rsn.beam_device_faults() == 0
