"""Attention over the 4-bit cache where units are cut between blocks and joined by the second kernel, against the plain
64-bit computation (needs a GB300).  Only cut units leave parts in the workspace, so that a case shows by it that it
took this way."""
import pytest
import torch

import residual_stream_norm_gb300 as rsn
from tests import _draft_ref as ref
from tests._gpu import Guarded, lib
from tests.test_gpu_kv4 import D, make

pytestmark = pytest.mark.gpu


def check(c, window=0, n_sink=0, sm_scale=None):
    B, N = c["table"].shape
    T, n_q, _ = c["q"].shape
    n = rsn.beam_attn_kv4_workspace(B, c["q_len"], n_q, c["k_cache"].shape[1], N, window, n_sink)
    ws = Guarded((n // 4,), dtype=torch.float32)
    ws.view.fill_(float("nan"))
    out, lse = Guarded((T, n_q, D)), Guarded((T, n_q), dtype=torch.float32)
    d = {x: c[x].cuda() for x in ("q", "k_cache", "v_cache", "k_scales", "v_scales", "table", "lens")}
    rsn.beam_attn_kv4_fwd(out.view, d["q"], d["k_cache"], d["v_cache"], d["k_scales"], d["v_scales"], d["table"],
                          d["lens"], ws.view.view(torch.uint8), group=c["group"], window=window, n_sink=n_sink,
                          sm_scale=sm_scale, lse_out=lse.view)
    torch.cuda.synchronize()
    for x in (ws, out, lse):
        x.check()
    assert not bool(torch.isnan(ws.view).all()), "no unit was cut"
    want, tol = ref.kv4_attention(c["q"], c["k_cache"], c["v_cache"], c["k_scales"], c["v_scales"], c["table"],
                                  c["lens"], c["q_len"], sm_scale, window, n_sink)
    o, z = out.view.cpu().double(), lse.view.cpu().double()
    empty = want[1] == -float("inf")
    assert torch.equal(empty, z == -float("inf")) and bool((o[empty] == 0).all())
    d = (o - want[0]).abs()
    assert bool((d <= tol[0]).all()), f"out: worst {float((d - tol[0]).max()):.3g} past the bound"
    d = (z - want[1])[~empty].abs()
    assert bool((d <= tol[1][~empty]).all()), f"lse: worst {float((d - tol[1][~empty]).max()):.3g}"


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("q_len,n_q,n_kv", [(1, 6, 1), (1, 12, 2), (2, 6, 1), (4, 6, 1), (3, 10, 2), (8, 6, 1)])
def test_row_tiles_and_groups(q_len, n_q, n_kv, group):
    lib()
    check(make(3, q_len, n_q, n_kv, [5001, 77, q_len], group, seed=q_len + n_q, S=6000))


@pytest.mark.parametrize("long", [0, 1, 299, 512, 699])
def test_more_sequences_than_a_block_has_threads(long):
    # several sequences to a thread that counts tiles, in front of the long one and behind it; some without keys
    lib()
    lens = [(i * 7) % 5 for i in range(700)]
    lens[long] = 10_001
    check(make(700, 1, 2, 1, lens, 128, seed=long, S=11_000))


def test_many_sequences_of_many_lengths():
    lib()
    lens = [(i * 37) % 97 for i in range(300)]
    lens[17], lens[200], lens[299] = 4000, 6500, 3000
    check(make(300, 2, 4, 2, lens, 64, seed=1, S=7000))


@pytest.mark.parametrize("window,n_sink", [(3000, 4), (3000, 70), (2017, 0), (1500, 1500)])
@pytest.mark.parametrize("q_len", [1, 4])
def test_windows_and_sinks(window, n_sink, q_len):
    lib()
    for group in (32, 128):
        check(make(4, q_len, 12, 2, [q_len, 7001, 3010, 1600], group, seed=window + n_sink, S=8000), window, n_sink)


def test_window_of_a_prompt_part():
    # row tiles that see different stretches of the list, each cut
    lib()
    check(make(1, 40, 6, 1, [6000], 64, seed=2), 2500, 30)


def test_slots_out_of_range():
    # single keys, whole tiles and all of a share without a slot; a sequence with none at all; keys only in the last tile
    lib()
    c = make(4, 2, 12, 2, [4000, 6001, 300, 2500], 64, seed=3, S=7000)
    S = c["k_cache"].shape[0]
    c["table"][0, ::3] = -1
    c["table"][0, 1000:1700] = S
    c["table"][1, 64:5900] = -(1 << 40)
    c["table"][2] = 1 << 33
    c["table"][3, :2470] = S + 5
    check(c)
    check(c, 2600, 9)


def test_lengths_past_the_table_and_padding():
    lib()
    c = make(5, 4, 6, 1, [5000, 2, 0, 4, 3000], 128, seed=4, S=6000)
    c["lens"][0], c["lens"][2] = 1 << 30, -7
    check(c)


def test_scores_that_rise_and_fall_along_a_list():
    # the parts' maxima differ by more than FP32's exponents hold
    lib()
    c = make(2, 1, 6, 1, [6000, 6000], 128, seed=5, S=12_100)
    at = c["table"][0]
    c["k_scales"][at, 0, 0] = torch.stack((0.3 * torch.linspace(0, 40, 6000), torch.zeros(6000)), 1).bfloat16()
    at = c["table"][1]
    c["k_scales"][at, 0, 0] = torch.stack((0.3 * torch.linspace(40, 0, 6000), torch.zeros(6000)), 1).bfloat16()
    check(c, sm_scale=0.3)


def test_one_head_in_a_wide_batch():
    # as many units as SMs, one of them long
    lib()
    lens = [3 + i % 11 for i in range(152)]
    lens[70] = 9000
    check(make(152, 1, 6, 1, lens, 128, seed=6, S=9500))
