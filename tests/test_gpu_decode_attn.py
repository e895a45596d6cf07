"""Attention over the slot cache with a shared prefix against a plain 64-bit computation (needs a
GB300).  The bounds count half a step of BF16 for the output, half a step of the weights' type for
each weight, and FP32 sums elsewhere."""
import math

import pytest
import torch

import residual_stream_norm_gb300 as rsn
from tests import _decode_ref as ref
from tests._gpu import CANARY, Guarded, lib

pytestmark = pytest.mark.gpu
D = 128


def make(B, q_len, n_q, n_kv, P, N, lens, fp8=False, seed=0, extra=7, q_pad=0, spread=1.0,
         page=0):
    """A case on the CPU: caches with distinct random slots (or pages of `page` consecutive ones), NaN in
    every slot that is not listed."""
    g = torch.Generator().manual_seed(seed)
    lens = [int(n) for n in lens]
    inside = [min(max(n, 0), N) for n in lens]
    total = P + sum(inside)
    S = total + extra
    perm = torch.randperm(S, generator=g)
    if page:
        S = -(-S // page) * page
        perm = (torch.randperm(S // page, generator=g)[:, None] * page + torch.arange(page)).view(-1)
    prefix = perm[:P].clone()
    table = torch.full((B, N), -1, dtype=torch.int64)
    at = P
    for b, n in enumerate(inside):
        table[b, :n] = perm[at:at + n]
        table[b, n:] = perm[total] if extra else -1  # what lies behind a length is never read
        at += n
    k = torch.randn((S, n_kv, D), generator=g) * spread
    v = torch.randn((S, n_kv, D), generator=g)
    ks, vs = 1.0, 1.0
    if fp8:
        ks, vs = 0.05, 0.03
        k = (k / ks).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        v = (v / vs).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        k[perm[total:]] = 0x7f
        v[perm[total:]] = 0xff
    else:
        k, v = k.bfloat16(), v.bfloat16()
        k[perm[total:]] = math.nan
        v[perm[total:]] = math.nan
    q = torch.randn((B * q_len, n_q + q_pad, D), generator=g).bfloat16()[:, :n_q]
    return dict(q=q, k=k, v=v, prefix=prefix, table=table,
                lens=torch.tensor(lens, dtype=torch.int32), q_len=q_len, ks=ks, vs=vs, fp8=fp8)


def run(c, window=0, weights=False, weight_in=None, sm_scale=None, out=None):
    B, N = c["table"].shape
    T, n_q, _ = c["q"].shape
    n_kv, P = c["k"].shape[1], c["prefix"].numel()
    dev = {x: c[x].cuda() for x in ("k", "v", "prefix", "table", "lens")}
    q = torch.empty_strided(c["q"].shape, c["q"].stride(), dtype=torch.bfloat16, device="cuda")
    q.copy_(c["q"])
    if out is None:
        out = Guarded((T, n_q, D))
    lse = Guarded((T, n_q), dtype=torch.float32)
    w = Guarded((B, N), dtype=torch.float32) if weights else None
    w_in = None if weight_in is None else weight_in.cuda()
    n = rsn.beam_attn_prefix_workspace(B, c["q_len"], n_q, n_kv, P, N, window, weights)
    # a workspace that holds NaN: nothing in it may be taken for data
    workspace = torch.full((n // 4 + 64,), math.nan, dtype=torch.float32, device="cuda")
    workspace[n // 4:] = CANARY
    used = workspace[:n // 4].view(torch.uint8)
    rsn.beam_attn_prefix_fwd(
        out.view, q, dev["k"], dev["v"], dev["prefix"], dev["table"], dev["lens"], used,
        cache_dtype=rsn.CACHE_FP8_E4M3 if c["fp8"] else rsn.CACHE_BF16, k_scale=c["ks"],
        v_scale=c["vs"], sm_scale=sm_scale, window=window, lse_out=lse.view,
        key_weight_out=None if w is None else w.view, key_weight_in=w_in)
    torch.cuda.synchronize()
    for x in (out, lse, w):
        if x is not None:
            x.check()
    assert bool((workspace[n // 4:] == CANARY).all()), "workspace overrun"
    return out.view.cpu(), lse.view.cpu(), None if w is None else w.view.cpu()


def check(c, window=0, weights=False, weight_in=None, sm_scale=None):
    got = run(c, window, weights, weight_in, sm_scale)
    want, tol = ref.attention(c["q"], c["k"], c["v"], c["prefix"], c["table"], c["lens"],
                              c["q_len"], c["ks"], c["vs"], sm_scale, window, weight_in, c["fp8"])
    for name, x, y, e in zip(("out", "lse", "weights"), got, want, tol):
        if x is None:
            continue
        x = x.double()
        inf = torch.isinf(y)
        assert bool((x[inf] == y[inf]).all()), name
        d = (x - y).abs()[~inf]
        bad = d > e[~inf]
        assert not bool(bad.any()) and bool(torch.isfinite(d).all()), \
            f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {float(d.max()):.3g}"
    return got


CASES = [
    # B, q_len, n_q, n_kv, P, N, lens
    (1, 1, 1, 1, 0, 1, [1]),                      # one key
    (1, 1, 6, 1, 0, 15, [15]),
    (1, 1, 48, 8, 0, 17, [17]),
    (2, 1, 6, 1, 1, 64, [64, 63]),
    (3, 1, 12, 2, 63, 65, [65, 1, 33]),
    (2, 1, 8, 8, 64, 130, [130, 127]),            # a KV head of its own for each query head
    (2, 1, 16, 1, 65, 200, [200, 77]),            # 16 rows a unit
    (1, 1, 40, 2, 129, 300, [300]),               # 20 query heads share a KV head
    (4, 1, 6, 1, 1000, 90, [0, 5, -3, 90]),       # padded sequences: rows that see nothing
    (2, 2, 6, 1, 0, 40, [1, 40]),                 # the first of two queries sees nothing
    (3, 4, 6, 1, 100, 70, [70, 4, 3]),
    (2, 7, 10, 2, 33, 50, [50, 8]),
    (1, 17, 6, 2, 40, 80, [80]),
    (2, 1, 6, 1, 50, 20, [25, 7]),                # a length past the table is limited to it
    (2, 1, 6, 1, 50, 0, [0, 0]),                  # no table at all
    (40, 1, 6, 1, 200, 9, list(range(1, 10)) * 4 + [9] * 4),  # many rows on the prefix
    (1, 1, 6, 1, 0, 3000, [2999]),                # many parts of one list
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_sizes(case, fp8):
    lib()
    B, q_len, n_q, n_kv, P, N, lens = case
    check(make(B, q_len, n_q, n_kv, P, N, lens, fp8=fp8, seed=B + N), weights=N > 0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [1, 8, 16, 24, 64, 10 ** 4])
def test_pages(page, fp8):
    # slots in runs of all lengths, which start and end inside the tiles; few and many prefix rows
    lib()
    check(make(3, 2, 12, 2, 300, 150, [150, 61, 16], fp8=fp8, seed=page, page=page), weights=True)
    check(make(3, 2, 6, 1, 300, 150, [150, 61, 16], fp8=fp8, seed=page, page=page), window=70)
    check(make(40, 1, 6, 1, 1000, 33, [1 + b % 33 for b in range(40)], fp8=fp8, seed=page,
               page=page))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [1, 16, 24])
def test_pages_on_a_long_prefix(page, fp8):
    lib()
    check(make(30, 1, 48, 8, 2500, 9, [1 + b % 9 for b in range(30)], fp8=fp8, seed=page, page=page))


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 200, 10 ** 12])
@pytest.mark.parametrize("P", [0, 100])
def test_windows(P, window):
    lib()
    check(make(3, 3, 6, 1, P, 150, [150, 70, 2], seed=window % 1000), window=window, weights=True)


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_slots_are_not_seen(fp8):
    lib()
    c = make(3, 1, 6, 2, 70, 100, [100, 40, 30], fp8=fp8, seed=3)
    S = c["k"].shape[0]
    c["prefix"][::7] = -1
    c["prefix"][3] = S
    c["table"][0, ::3] = -1
    c["table"][1, :40] = S + 5              # a sequence that sees prefix keys only
    c["table"][2, 5] = 2 ** 40
    c["table"][2, 6] = -2 ** 62
    check(c, weights=True)
    c["prefix"][:] = -1                     # and one that sees nothing at all
    out, lse, w = check(c, weights=True)
    assert bool((out[1] == 0).all()) and bool((lse[1] == -math.inf).all())


def test_accumulates_weights_in_place_and_strided():
    lib()
    c = make(2, 1, 12, 2, 30, 50, [50, 20], seed=5)
    w0 = torch.rand((2, 50))
    want, tol = ref.attention(c["q"], c["k"], c["v"], c["prefix"], c["table"], c["lens"], 1,
                              weight_in=w0)
    _, _, w = check(c, weights=True, weight_in=w0)
    assert torch.equal(w[1, 20:], w0[1, 20:])          # what lies behind a length is only copied
    wide = torch.zeros((2, 80), device="cuda")
    wide[:, :50] = w0.cuda()
    table = torch.full((2, 64), 2 ** 50, dtype=torch.int64, device="cuda")
    table[:, :50] = c["table"].cuda()
    n = rsn.beam_attn_prefix_workspace(2, 1, 12, 2, 30, 50, 0, True)
    out = torch.empty_like(c["q"], device="cuda")
    rsn.beam_attn_prefix_fwd(out, c["q"].cuda(), c["k"].cuda(), c["v"].cuda(), c["prefix"].cuda(),
                             table[:, :50], c["lens"].cuda(),
                             torch.empty(n, dtype=torch.uint8, device="cuda"),
                             key_weight_in=wide[:, :50], key_weight_out=wide[:, :50])
    torch.cuda.synchronize()
    assert torch.equal(wide[:, :50].cpu(), w)
    assert bool((wide[:, 50:] == 0).all())


def test_strided_query_and_output_rows():
    lib()
    c = make(3, 2, 6, 1, 40, 60, [60, 33, 2], seed=6, q_pad=3)
    assert not c["q"].is_contiguous()
    plain = check(c)[0]
    wide = Guarded((6, 9, D))
    view = wide.view
    wide.view = view[:, 1:7]
    got = run(c, out=wide)[0]
    assert torch.equal(got, plain)
    assert bool((view[:, 0] == CANARY).all()) and bool((view[:, 7:] == CANARY).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_peaked_scores_and_scales(fp8):
    # scores up to several hundred: one key takes nearly all the weight
    lib()
    c = make(2, 1, 12, 2, 130, 140, [140, 90], fp8=fp8, seed=8, spread=8.0)
    check(c, weights=True, sm_scale=1.0)
    check(c, sm_scale=-0.3)
    check(c, sm_scale=0.0)


def test_fp8_query_range():
    # rows of very large, very small and zero queries: the FP16 scaling is by row
    lib()
    c = make(4, 1, 6, 1, 20, 30, [30, 30, 12, 1], fp8=True, seed=9)
    c["q"][0] *= 2.0 ** 100
    c["q"][1] *= 2.0 ** -100
    c["q"][2] = 0
    check(c, sm_scale=2.0 ** -100)
    c["q"][0] *= 2.0 ** -100
    check(c, sm_scale=0.1)


def test_non_finite_inputs_stay_in_their_rows():
    lib()
    c = make(3, 1, 6, 1, 40, 50, [50, 50, 50], seed=10)
    clean = run(c)[0]
    c["k"][c["table"][0, 3], 0, 5] = math.nan
    c["v"][c["table"][1, 7], 0, 9] = math.inf
    out, lse, _ = run(c)
    assert bool(torch.isnan(out[0]).all()) and bool(torch.isnan(lse[0]).all())
    assert bool((out[1, :, 9] == math.inf).all())
    assert torch.equal(out[1, :, :9], clean[1, :, :9]) and torch.equal(out[2], clean[2])


def test_values_of_unseen_keys_do_not_matter():
    # a later token's or an out-of-window key's value may be NaN or infinite
    lib()
    c = make(2, 4, 6, 1, 30, 60, [60, 45], seed=11)
    clean = run(c, window=20)[0]
    for b, n in ((0, 60), (1, 45)):
        c["v"][c["table"][b, n - 1], 0] = math.nan   # the last token: seen by the last query only
        c["v"][c["table"][b, n - 2], 0, 3] = -math.inf
        c["v"][c["table"][b, n - 23], 0] = math.nan  # out of the window of the last query only
    out = run(c, window=20)[0].view(2, 4, 6, D)
    clean = clean.view(2, 4, 6, D)
    assert torch.equal(out[:, 1], clean[:, 1])
    assert bool(torch.isnan(out[:, 3]).all()) and bool(torch.isnan(out[:, 0]).all())
    assert bool((out[:, 2, :, 3] == -math.inf).all())
    assert torch.equal(out[:, 2, :, 4:], clean[:, 2, :, 4:])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,P,window", [(30, 3000, 2700), (20, 4600, 4200)])
def test_values_that_a_window_hides_from_some_rows(B, P, window, fp8):
    # prefix values that are not finite: rows that see them show it, the others do not change
    lib()
    lens = [1 + 7 * b for b in range(B)]
    c = make(B, 1, 48, 8, P, 7 * B, lens, fp8=fp8, seed=B)
    clean = run(c, window=window)[0]
    j = P - window + 60                        # out of the window of the longer sequences
    c["v"][c["prefix"][j], 3, 9] = 0x7f if fp8 else math.nan
    if not fp8:
        c["v"][c["prefix"][j + 1], 3, 5] = -math.inf
    out = run(c, window=window)[0]
    for b, n in enumerate(lens):
        sees, sees1 = n - 1 < window - P + j, n - 1 < window - P + j + 1
        assert bool(torch.isnan(out[b, 18:24, 9]).all()) == sees, b
        if not fp8:
            assert bool((out[b, 18:24, 5] == -math.inf).all()) == sees1, b
        keep = [d for d in range(D) if d not in (5, 9)]
        assert torch.equal(out[b][:, keep], clean[b][:, keep]), b
        assert torch.equal(out[b, :18], clean[b, :18]) and torch.equal(out[b, 24:], clean[b, 24:]), b


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,q_len,n_q,n_kv,P,window", [
    (43, 1, 48, 8, 2000, 0), (20, 1, 48, 8, 4001, 0), (13, 5, 48, 8, 2500, 0),
    (25, 2, 48, 8, 2600, 1800), (20, 1, 48, 8, 4000, 3900), (3, 1, 48, 8, 20000, 0),
    (60, 1, 40, 8, 1300, 0)])
def test_many_rows_on_a_long_prefix(B, q_len, n_q, n_kv, P, window, fp8):
    # enough work for the kernel for many prefix rows, with ragged row and key tiles and padded rows
    lib()
    lens = [(7 * b) % 12 for b in range(B)]
    check(make(B, q_len, n_q, n_kv, P, 11, lens, fp8=fp8, seed=P), window=window, weights=True)


@pytest.mark.parametrize("fp8", [False, True])
def test_long_prefix_with_bad_slots(fp8):
    lib()
    c = make(25, 1, 48, 8, 3000, 5, [5] * 25, fp8=fp8, seed=4)
    c["prefix"][::9] = -1
    c["prefix"][1:2500:250] = c["k"].shape[0]
    c["prefix"][700:1100] = 2 ** 45
    check(c)


def test_same_bits_every_time_and_on_another_stream():
    lib()
    c = make(20, 1, 48, 8, 500, 200, [200 - 9 * b for b in range(20)], seed=13)
    first = run(c, weights=True)
    for _ in range(3):
        again = run(c, weights=True)
        assert all(torch.equal(x, y) for x, y in zip(first, again))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        again = run(c, weights=True)
    assert all(torch.equal(x, y) for x, y in zip(first, again))


def test_graph_replay_reads_the_lengths_anew():
    lib()
    c = make(4, 1, 6, 1, 100, 80, [80, 80, 80, 80], seed=14)
    want_full = run(c)[0]
    dev = {x: c[x].cuda() for x in ("q", "k", "v", "prefix", "table", "lens")}
    out = torch.zeros_like(dev["q"])
    n = rsn.beam_attn_prefix_workspace(4, 1, 6, 1, 100, 80)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def call():
        rsn.beam_attn_prefix_fwd(out, dev["q"], dev["k"], dev["v"], dev["prefix"], dev["table"],
                                 dev["lens"], ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want_full)
    c["lens"] = torch.tensor([1, 17, 0, 64], dtype=torch.int32)
    want = run(c)[0]
    dev["lens"].copy_(c["lens"])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want)


def test_cache_offsets_past_32_bits():
    lib()
    S = 2_200_000                                     # 4.5 GB a cache
    k = torch.zeros((S, 8, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    c = make(2, 1, 48, 8, 50, 40, [40, 23], seed=15, extra=1)
    n = c["k"].shape[0]
    k[-n:] = c["k"].cuda()
    v[-n:] = c["v"].cuda()
    want = run(c)[0]
    out = torch.empty_like(want, device="cuda")
    ws = torch.empty(rsn.beam_attn_prefix_workspace(2, 1, 48, 8, 50, 40), dtype=torch.uint8,
                     device="cuda")
    rsn.beam_attn_prefix_fwd(out, c["q"].cuda(), k, v, (c["prefix"] + S - n).cuda(),
                             (c["table"] + S - n).cuda(), c["lens"].cuda(), ws)
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want)


def test_zero_sequences():
    lib()
    e = torch.empty
    rsn.beam_attn_prefix_fwd(
        e((0, 6, D), dtype=torch.bfloat16, device="cuda"),
        e((0, 6, D), dtype=torch.bfloat16, device="cuda"),
        e((3, 1, D), dtype=torch.bfloat16, device="cuda"),
        e((3, 1, D), dtype=torch.bfloat16, device="cuda"), None,
        e((0, 4), dtype=torch.int64, device="cuda"), e((0,), dtype=torch.int32, device="cuda"),
        e((1,), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("graph", [False, True])
def test_right_behind_the_kernels_that_write_its_inputs(graph, fp8):
    # a long prefix for many rows; Q/K norm writes the queries and the newest keys and values, eviction the
    # table, lengths and weights, and attention follows at once
    lib()
    B, n_q, n_kv, P, width, budget = 25, 48, 8, 3000, 9, 6
    g = torch.Generator().manual_seed(16)
    ks, vs = (0.05, 0.03) if fp8 else (1.0, 1.0)
    S = P + B * width
    perm = torch.randperm(S, generator=g)
    prefix, own = perm[:P].cuda(), perm[P:].view(B, width).cuda()
    caches = []
    for scale in (ks, vs):
        x = torch.randn((S, n_kv, D), generator=g)
        x = (x / scale).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else x.bfloat16()
        caches.append(x.cuda())
    k, v = caches
    wq, wk = (torch.ones(D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pos = torch.full((B,), P + width - 1, dtype=torch.int64, device="cuda")
    tokens = torch.randn((4, B, n_q + 2 * n_kv, D), generator=g).bfloat16().cuda()
    weights = torch.rand((4, B, width), generator=g).cuda()
    qkv, w = torch.empty_like(tokens[0]), torch.empty_like(weights[0])
    q, k_new, v_new = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
    slots = own[:, -1].contiguous()
    table, lens = own.clone(), torch.full((B,), width, dtype=torch.int32, device="cuda")
    freed = torch.empty((B, width - budget), dtype=torch.int64, device="cuda")
    out = torch.empty((B, n_q, D), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((B, n_q), dtype=torch.float32, device="cuda")
    ws = torch.empty(rsn.beam_attn_prefix_workspace(B, 1, n_q, n_kv, P, width, key_weights=True),
                     dtype=torch.uint8, device="cuda")
    kind = rsn.CACHE_FP8_E4M3 if fp8 else rsn.CACHE_BF16

    def attend(out, lse, w_in, w_out):
        rsn.beam_attn_prefix_fwd(out, q, k, v, prefix, table, lens, ws, cache_dtype=kind, k_scale=ks,
                                 v_scale=vs, lse_out=lse, key_weight_in=w_in, key_weight_out=w_out)

    def steps():
        rsn.beam_kv_evict_fwd(table, lens, w, freed, table, lens, w, budget, 2)
        rsn.beam_qk_norm_ssmax_kv_fwd(q, k_new, v_new, wq, wk, pos, slots, k, v, cache_dtype=kind,
                                      k_scale=ks, v_scale=vs)
        attend(out, lse, w, w)

    def inputs(i):
        qkv.copy_(tokens[i])
        w.copy_(weights[i])
        table.copy_(own)
        lens.fill_(width)

    if graph:
        inputs(0)
        steps()
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            steps()
    for i in range(4):
        inputs(i)
        captured.replay() if graph else steps()
        torch.cuda.synchronize()
        # what the writers left, and attention over it once more, by itself
        kept, n, w0, _ = ref.evict(own.cpu().numpy(), [width] * B, weights[i].cpu().numpy(), budget, 2,
                                   width - budget)
        w0 = torch.from_numpy(w0)
        assert torch.equal(table.cpu(), torch.from_numpy(kept)) and bool((lens == budget).all())
        again = [torch.empty_like(x) for x in (out, lse, w)]
        attend(again[0], again[1], w0.cuda(), again[2])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((out, lse, w), again))
    want, tol = ref.attention(q.cpu(), k.cpu(), v.cpu(), prefix.cpu(), table.cpu(), lens.cpu(), 1, ks,
                              vs, weight_in=w0, fp8=fp8)
    for x, y, e in zip((out, lse, w), want, tol):
        assert bool(((x.cpu().double() - y).abs() <= e).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,P,N", [
    (1, 0, 2001),        # a sequence's own keys
    (2, 100, 2001),      # behind a prefix in line
    (8, 40001, 1),       # a prefix for up to 128 rows on the tensor cores
    (9, 50001, 1)])      # and for more
def test_small_weights_beside_strong_keys(B, P, N, fp8):
    # every sixteenth key takes nearly all of the weight and has no value: the output is what the others,
    # each of 1.4 x 2^-24 of a strong key's weight, add up to
    lib()
    n_q, S = 16, P + B * N
    strong = torch.arange(S) % 16 == 0
    k = torch.zeros((S, 1, D))
    k[strong, 0, 0] = 1.0
    v = torch.ones((S, 1, D))
    v[strong] = 0.0
    q = torch.zeros((B, n_q, D), dtype=torch.bfloat16)
    q[:, :, 0] = 1.0
    cast = (lambda x: x.to(torch.float8_e4m3fn).view(torch.uint8)) if fp8 else (
        lambda x: x.bfloat16())
    c = dict(q=q, k=cast(k), v=cast(v), prefix=torch.arange(P), table=P + torch.arange(B * N).view(B, N),
             lens=torch.full((B,), N, dtype=torch.int32), q_len=1, ks=1.0, vs=1.0, fp8=fp8)
    sm = 24 * math.log(2.0) - math.log(1.4)
    out, lse, w = run(c, weights=True, sm_scale=sm)
    # a sequence's rows are alike: one of each in 64 bits
    for b in range(B):
        want, tol = ref.attention(q[:1, :1], c["k"], c["v"], c["prefix"], c["table"][b:b + 1],
                                  c["lens"][:1], 1, sm_scale=sm, fp8=fp8)
        assert float(tol[0].max()) < 0.02 * float(want[0].min())
        assert bool(((out[b].double() - want[0][0]).abs() <= tol[0][0]).all()), \
            f"{out[b].min():.4g} to {out[b].max():.4g} for {float(want[0].min()):.4g}"
        assert bool(((lse[b].double() - want[1][0]).abs() <= tol[1][0]).all())
        assert bool(((w[b].double() - n_q * want[2][0]).abs() <= n_q * tol[2][0]).all())


def test_one_long_list_among_many_short_ones():
    # the long list is shared out: the call takes little more than its two parts by themselves (all of a head's
    # 60,000 keys in one block would take some ten times as long)
    lib()
    B, n = 256, 60000
    short = [1 + (37 * b) % 200 for b in range(B)]
    times = []
    for lens, N in ((short, n), ([n], n), (short[:90] + [n] + short[91:], n)):
        c = make(len(lens), 1, 8, 8, 0, N, lens, seed=17)
        dev = {x: c[x].cuda() for x in ("q", "k", "v", "table", "lens")}
        ws = torch.empty(rsn.beam_attn_prefix_workspace(len(lens), 1, 8, 8, 0, N), dtype=torch.uint8,
                         device="cuda")
        out = torch.empty_like(dev["q"])
        best = math.inf
        for _ in range(8):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            rsn.beam_attn_prefix_fwd(out, dev["q"], dev["k"], dev["v"], None, dev["table"], dev["lens"],
                                     ws)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        times.append(best)
    assert times[2] < 3 * (times[0] + times[1]), times
    pick = [0, 90, 200]
    want, tol = ref.attention(c["q"][pick], c["k"], c["v"], c["prefix"], c["table"][pick],
                              c["lens"][pick], 1)
    assert bool(((out.cpu()[pick].double() - want[0]).abs() <= tol[0]).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,n_q,n_kv,P,N", [
    (129, 6, 1, 0, 150),    # the last sequence starts a second round of the sums over the sequences
    (300, 6, 1, 0, 150),
    (300, 4, 2, 300, 90),   # with a prefix in units of its own or on the tensor cores
    (260, 8, 8, 0, 200)])   # whole units of several tiles
def test_more_sequences_than_threads_of_a_block(B, n_q, n_kv, P, N, fp8):
    lib()
    lens = [(53 * b) % (N + 1) for b in range(B)]
    for b in (0, 126, 127, 128, 255, 256, B - 1):       # without a key, around the rounds' ends
        if b < B:
            lens[b] = 0
    lens[1], lens[125], lens[B - 2] = N, N, N
    c = make(B, 1, n_q, n_kv, P, N, lens, fp8=fp8, seed=B + n_q)
    plain = check(c, weights=True)
    assert all(torch.equal(x, y) for x, y in zip(run(c), plain[:2]))  # with and without weights
    check(c, window=77)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,P,N", [(7, 0, 1), (3, 0, 3000)])
def test_log_sums_near_zero(B, P, N, fp8):
    # sums next to 1 (one key, or a strong one among weak ones): a few steps of FP32 at 1, whatever the weights
    # are scaled by
    lib()
    c = make(B, 1, 8, 8, P, N, [N] * B, fp8=fp8, seed=18)
    c["q"] *= 0.125
    c["k"][c["table"][:, 1:].flatten()] = 0
    if N > 1:
        c["q"][:] = 0
        c["q"][:, :, 0] = 1.0
        c["k"][c["table"][:, 1:].flatten(), :, 0] = 0xfe if fp8 else -448.0  # the lowest E4M3 number
        c["k"][c["table"][:, 0]] = 0
    sm = 0.0625
    ks = c["ks"] if fp8 else 1.0
    _, lse, _ = run(c, sm_scale=sm, weights=True)
    for b in range(B):
        kk = ref.cache_values(c["k"][c["table"][b]], ks).transpose(0, 1)          # [8, N, D]
        s = torch.einsum("hd,hnd->hn", c["q"][b].double(), kk) * sm
        want = torch.logsumexp(s, 1)
        # the score's rounding (as in the reference), one of exp2 and two of the logarithm near 1, one of the sum
        tol = (c["q"][b].double().abs()[:, None] * kk.abs()).sum(2).max() * sm * 128 * ref.U32 * 2 + \
            (8 * s.abs().max(1).values.clamp(min=1.0)) * ref.U32
        assert bool(((lse[b].double() - want).abs() <= tol).all()), (lse[b], want)
