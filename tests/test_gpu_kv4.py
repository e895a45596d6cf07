"""The KV cache held in 4 bits: its write (equal bit for bit) and its attention against plain 64-bit
computations, with bounds that count half a step of each rounded type (needs a GB300)."""
import pytest
import torch

import residual_stream_norm_gb300 as rsn
from tests import _draft_ref as ref
from tests._gpu import Guarded, lib

pytestmark = pytest.mark.gpu
D = 128


# ---------------------------------------------------------------------------------------------
# write
# ---------------------------------------------------------------------------------------------

def cache(S, n_kv, group, fill=True):
    g = torch.Generator().manual_seed(S)
    c = [torch.randint(0, 256, (S, n_kv, 64), generator=g, dtype=torch.uint8) for _ in range(2)]
    s = [torch.randn((S, n_kv, D // group, 2), generator=g).bfloat16() for _ in range(2)]
    return c + s


def run_write(k, v, slots, S, group):
    kc, vc, ks, vs = (t.cuda() for t in cache(S, k.shape[1], group))
    rsn.beam_kv4_write_fwd(kc, vc, ks, vs, k, v, slots.cuda(), group=group)
    torch.cuda.synchronize()
    return [t.cpu() for t in (kc, vc, ks, vs)]


def check_write(k, v, slots, S, group, kd=None, vd=None):
    got = run_write(k.cuda() if kd is None else kd, v.cuda() if vd is None else vd, slots, S, group)
    want = cache(S, k.shape[1], group)
    on = (slots >= 0) & (slots < S)
    for i, x in ((0, k), (1, v)):
        codes, scales = ref.kv4_write(x, group)
        want[i][slots[on]] = codes[on]
        want[i + 2][slots[on]] = scales[on]
    for a, b in zip(got[:2], want[:2]):
        assert torch.equal(a, b)
    for a, b in zip(got[2:], want[2:]):
        assert torch.equal(torch.nan_to_num(a, nan=-77.0), torch.nan_to_num(b, nan=-77.0))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,n_kv", [(1, 1), (1, 8), (2, 3), (7, 5), (33, 2), (150, 8)])
def test_write_sizes(T, n_kv, group):
    lib()
    g = torch.Generator().manual_seed(T)
    k, v = (torch.randn((T, n_kv, D), generator=g).bfloat16() for _ in range(2))
    k[:, :, 3] *= 9
    slots = torch.randperm(T + 40, generator=g)[:T]
    slots[T // 2] = -1 if T % 2 else T + 40
    check_write(k, v, slots, T + 40, group)


def test_write_strided_rows():
    lib()
    x = torch.randn((9, 10, D), generator=torch.Generator().manual_seed(2)).bfloat16()
    xd = x.cuda()
    check_write(x[:, 6:8], x[:, 8:], torch.randperm(30)[:9], 30, 64, xd[:, 6:8], xd[:, 8:])


def test_write_values_where_it_can_go_wrong():
    # flat rows, zeros of both signs, one far value, tiny and huge ones, NaN and infinities by group
    lib()
    inf, nan = float("inf"), float("nan")
    k = torch.randn((10, 2, D), generator=torch.Generator().manual_seed(3)).bfloat16()
    k[0] = 1.5
    k[1] = 0.0
    k[1, 0, ::2] = -0.0
    k[2, 0, 7] = 3.0e4
    k[3] *= 1e-38
    k[4] *= 1e37
    k[5, 0, 40] = nan
    k[5, 1, 100] = inf
    k[6, 0, 0] = -inf
    k[7, 0, 0], k[7, 0, 1] = 3.0e38, -3.0e38
    k[8] = torch.arange(D).float().bfloat16()
    k[9, 0] = torch.arange(D).remainder(16).bfloat16()
    for group in (32, 64, 128):
        check_write(k, k.flip(0), torch.arange(10), 10, group)


def test_write_nothing():
    lib()
    e = torch.empty((0, 2, D), dtype=torch.bfloat16)
    check_write(e, e, torch.empty(0, dtype=torch.int64), 5, 128)


# ---------------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------------

def make(B, q_len, n_q, n_kv, lens, group, seed=0, width=None, S=None):
    g = torch.Generator().manual_seed(seed)
    lens = torch.tensor(lens, dtype=torch.int32)
    N = max(1, int(lens.max())) if width is None else width
    S = B * N + 7 if S is None else S
    kc, vc = (torch.randint(0, 256, (S, n_kv, 64), generator=g, dtype=torch.uint8) for _ in range(2))
    ks, vs = (torch.stack((0.1 + 0.2 * torch.rand((S, n_kv, D // group), generator=g),
                           -1.6 - torch.rand((S, n_kv, D // group), generator=g)), 3).bfloat16()
              for _ in range(2))
    table = torch.randperm(S, generator=g)[:B * N].view(B, N) if B * N <= S else \
        torch.randint(0, S, (B, N), generator=g)
    q = torch.randn((B * q_len, n_q, D), generator=g).bfloat16()
    return dict(q=q, k_cache=kc, v_cache=vc, k_scales=ks, v_scales=vs, table=table, lens=lens, q_len=q_len,
                group=group)


def run(c, window=0, n_sink=0, sm_scale=None, qd=None, out=None, d=None):
    B, N = c["table"].shape
    T, n_q, _ = c["q"].shape
    d = d or {x: c[x].cuda() for x in ("k_cache", "v_cache", "k_scales", "v_scales", "table", "lens")}
    n = rsn.beam_attn_kv4_workspace(B, c["q_len"], n_q, c["k_cache"].shape[1], N, window, n_sink)
    ws = Guarded((max(16, n) // 4 + 1,), dtype=torch.float32)
    ws.view.fill_(float("nan"))
    out = out or Guarded((T, n_q, D))
    lse = Guarded((T, n_q), dtype=torch.float32)
    rsn.beam_attn_kv4_fwd(out.view, c["q"].cuda() if qd is None else qd, d["k_cache"], d["v_cache"],
                          d["k_scales"], d["v_scales"], d["table"], d["lens"],
                          ws.view.view(torch.uint8), group=c["group"], window=window, n_sink=n_sink,
                          sm_scale=sm_scale, lse_out=lse.view)
    torch.cuda.synchronize()
    for x in (ws, out, lse):
        x.check()
    return out.view.cpu(), lse.view.cpu()


def check(c, window=0, n_sink=0, sm_scale=None, **kw):
    out, lse = run(c, window, n_sink, sm_scale, **kw)
    want, tol = ref.kv4_attention(c["q"], c["k_cache"], c["v_cache"], c["k_scales"], c["v_scales"], c["table"],
                                  c["lens"], c["q_len"], sm_scale, window, n_sink)
    d = (out.double() - want[0]).abs()
    assert bool((d <= tol[0]).all()), f"out: worst {float((d - tol[0]).max()):.3g} past the bound"
    empty = want[1] == -float("inf")
    assert torch.equal(empty, lse == -float("inf")) and bool((out[empty] == 0).all())
    d = (lse.double() - want[1])[~empty].abs()
    assert bool((d <= tol[1][~empty]).all()), f"lse: worst {float((d - tol[1][~empty]).max()):.3g}"
    return out, lse


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("q_len,n_q,n_kv", [(1, 48, 8), (1, 1, 1), (1, 8, 8), (2, 12, 2), (4, 6, 1),
                                            (1, 16, 1), (3, 10, 2), (8, 12, 2), (5, 40, 8), (1, 64, 1)])
def test_heads_and_groups(q_len, n_q, n_kv, group):
    lib()
    check(make(3, q_len, n_q, n_kv, [q_len, 70, 131], group, seed=q_len + n_q))


@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200])
def test_lengths(n):
    lib()
    check(make(2, 1, 6, 1, [n, 64], 128, seed=n, width=210))
    check(make(2, 3, 6, 1, [n, 5], 64, seed=n, width=210))


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (5, 2), (64, 4), (64, 64), (100, 70), (512, 4),
                                           (150, 0), (1000, 3)])
@pytest.mark.parametrize("q_len", [1, 4])
def test_window_and_sinks(window, n_sink, q_len):
    lib()
    check(make(4, q_len, 12, 2, [q_len, 66, 170, 333], 128, seed=window), window, n_sink)
    check(make(2, q_len, 12, 2, [3, 257], 32, seed=window), window, n_sink)


def test_padding_and_lengths_out_of_range():
    lib()
    c = make(5, 4, 6, 1, [0, 2, 4, 50, 60], 128, seed=1)
    c["lens"][0], c["lens"][4] = -3, 10_000
    check(c)


def test_slots_out_of_range():
    # keys without a slot are not seen, wherever they stand; also a sequence that has none at all
    lib()
    c = make(3, 2, 12, 2, [80, 130, 20], 64, seed=2)
    S = c["k_cache"].shape[0]
    c["table"][0, ::3] = -1
    c["table"][1, 64:] = S + 5
    c["table"][2] = -(1 << 40)
    check(c)
    check(c, window=17, n_sink=3)


def test_no_slots_at_all():
    lib()
    c = make(2, 1, 6, 1, [3, 4], 128, S=20)
    for x in ("k_cache", "v_cache", "k_scales", "v_scales"):
        c[x] = c[x][:0]
    check(c)


def test_unseen_keys_leave_no_trace():
    # NaN, infinite and huge scales and minima in keys that a row does not see: those of other sequences,
    # those behind its own place, those between sinks and window
    lib()
    c = make(3, 3, 12, 2, [70, 9, 200], 32, seed=5)
    clean = run(c, window=40, n_sink=4)
    inf, nan = float("inf"), float("nan")
    bad = torch.tensor([[nan, nan], [inf, inf], [1.0, -inf], [3.0e38, 3.0e38], [nan, 0.0]]).bfloat16()
    own = [c["table"][b, :int(n)] for b, n in enumerate(c["lens"])]
    seen_later = torch.stack([o[-1:] for o in own]).flatten()           # only each last row sees these
    hidden = torch.cat((own[2][4:150], torch.tensor([3])))
    hidden = hidden[~torch.isin(hidden, torch.cat(own[:2]))]
    for i, s in enumerate(hidden.tolist()):
        c["k_scales"][s] = bad[i % 5]
        c["v_scales"][s] = bad[(i + 2) % 5]
    got = run(c, window=40, n_sink=4)
    assert all(torch.equal(a, b) for a, b in zip(got, clean))
    for i, s in enumerate(seen_later.tolist()):
        c["k_scales"][s, :, 1] = nan
        c["v_scales"][s] = bad[i]
    out, lse = run(c, window=40, n_sink=4)
    rows = torch.arange(9).view(3, 3)
    for a, b in ((out, clean[0]), (lse, clean[1])):
        # a row's masked keys may move its power-of-two reference, never its values beyond a rounding
        first = rows[:, :2].flatten()
        assert torch.equal(a[first], b[first])
        assert bool(torch.isnan(a[rows[:, 2]]).all())


def test_nan_key_shows():
    lib()
    c = make(1, 1, 6, 1, [100], 128, seed=6)
    c["v_scales"][c["table"][0, 30], 0, 0, 0] = float("nan")
    out, lse = run(c)
    assert bool(torch.isnan(out).all()) and bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("scale", [1e-30, 1e-6, 1e6, 1e30])
def test_scales_of_any_size(scale):
    lib()
    c = make(2, 1, 6, 1, [65, 150], 64, seed=7)
    c["v_scales"] = (c["v_scales"].float() * scale).bfloat16()
    check(c)
    c["v_scales"][::5] = (c["v_scales"][::5].float() * 1e-5).bfloat16()
    c["v_scales"][::7, :, 1] = 0
    check(c)


def test_flat_and_zero_rows():
    lib()
    c = make(2, 1, 6, 1, [65, 150], 128, seed=8)
    c["v_scales"][..., 0] = 0
    check(c)
    c["k_scales"][...] = 0
    check(c)
    c["q"][...] = 0
    check(c)


@pytest.mark.parametrize("sm_scale", [1.0, 0.0, -0.1, 3.0])
def test_scale_of_the_scores(sm_scale):
    lib()
    check(make(2, 2, 6, 1, [40, 140], 128, seed=9), sm_scale=sm_scale)


def test_large_and_uneven_queries():
    lib()
    c = make(2, 1, 6, 1, [40, 140], 128, seed=10)
    c["q"][0] = (c["q"][0].float() * 1e4).bfloat16()
    c["q"][1] = (c["q"][1].float() * 2.0 ** -60).bfloat16()
    c["q"][1, :, 0] = 1.0
    check(c, sm_scale=1e-3)


def test_strided_rows_and_wide_tables():
    lib()
    c = make(4, 1, 12, 2, [10, 66, 100, 0], 64, seed=11, width=120)
    plain = check(c)
    packed = torch.randn((4, 20, D)).bfloat16().cuda()
    packed[:, 3:15] = c["q"].cuda()
    wide = torch.full((4, 300), -9, dtype=torch.int64, device="cuda")
    wide[:, 50:170] = c["table"].cuda()
    d = {x: c[x].cuda() for x in ("k_cache", "v_cache", "k_scales", "v_scales", "lens")}
    d["table"] = wide[:, 50:170]
    out = Guarded((4, 20, D))
    full = out.view.fill_(5.0)
    out.view = full[:, 2:14]
    got = run(c, qd=packed[:, 3:15], out=out, d=d)
    assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])
    assert bool((full[:, :2] == 5).all()) and bool((full[:, 14:] == 5).all())


def test_many_sequences():
    # more sequences than a block has threads, most of them short or empty, one long
    lib()
    lens = [(i * 7) % 5 for i in range(700)]
    lens[333] = 3001
    check(make(700, 1, 2, 1, lens, 128, seed=12, S=4000))


def test_long_list_cut_between_all_warps():
    lib()
    check(make(1, 1, 6, 1, [90_001], 128, seed=13))
    check(make(2, 4, 6, 1, [40_000, 64], 32, seed=14, S=50_000))


def test_offsets_past_32_bits():
    # slots at the end of a cache of more than 4 GiB
    lib()
    S, n_kv = 8_500_000, 8
    c = make(2, 1, 8, n_kv, [70, 130], 128, seed=15)
    n = c["k_cache"].shape[0]
    d = {x: torch.zeros((S,) + c[x].shape[1:], dtype=c[x].dtype, device="cuda")
         for x in ("k_cache", "v_cache", "k_scales", "v_scales")}
    for x in d:
        d[x][S - n:] = c[x].cuda()
    d["table"], d["lens"] = c["table"].cuda() + (S - n), c["lens"].cuda()
    want = run(c)
    got = run(c, d=d)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    k, v = (torch.randn((3, n_kv, D)).bfloat16() for _ in range(2))
    slots = torch.tensor([S - 1, S - 9, 4])
    rsn.beam_kv4_write_fwd(d["k_cache"], d["v_cache"], d["k_scales"], d["v_scales"], k.cuda(), v.cuda(),
                           slots.cuda())
    for x, i in (("k", k), ("v", v)):
        codes, scales = ref.kv4_write(i, 128)
        assert torch.equal(d[x + "_cache"][slots.cuda()].cpu(), codes)
        assert torch.equal(d[x + "_scales"][slots.cuda()].cpu(), scales)


def test_same_bits_every_time_and_in_a_graph():
    lib()
    c = make(9, 2, 12, 2, [5, 900, 64, 0, 333, 2000, 1, 77, 1500], 64, seed=16)
    first = run(c)
    assert all(torch.equal(a, b) for _ in range(3) for a, b in zip(run(c), first))
    d = {x: c[x].cuda() for x in ("q", "k_cache", "v_cache", "k_scales", "v_scales", "table", "lens")}
    ws = torch.empty(rsn.beam_attn_kv4_workspace(9, 2, 12, 2, 2000), dtype=torch.uint8, device="cuda")
    out = torch.zeros((18, 12, D), dtype=torch.bfloat16, device="cuda")

    def call():
        rsn.beam_attn_kv4_fwd(out, d["q"], d["k_cache"], d["v_cache"], d["k_scales"], d["v_scales"],
                              d["table"], d["lens"], ws, group=64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        out.fill_(7)
        graph.replay()
        assert torch.equal(out.cpu(), first[0])
    # the lengths are read when the graph runs
    d["lens"].fill_(3)
    graph.replay()
    c["lens"][:] = 3
    assert torch.equal(out.cpu(), run(c)[0])


def test_more_query_rows_than_warps():
    # more KV heads and row tiles than an SM's, and than all SMs' warps (whole units, and one cut by its rows alone)
    lib()
    check(make(2, 150, 16, 2, [200, 40], 64, seed=18))
    check(make(1, 500, 64, 8, [1500], 128, seed=19))


def test_windows_past_the_table():
    lib()
    c = make(3, 2, 12, 2, [2, 70, 300], 64, seed=20)
    plain = run(c)
    for window, n_sink in ((1 << 62, 0), (300, 5), (7, 1 << 62)):
        assert all(torch.equal(a, b) for a, b in zip(run(c, window, n_sink), plain))


def test_no_table_at_all():
    lib()
    c = make(2, 3, 6, 1, [0, 0], 128, width=1)
    c["table"] = c["table"][:, :0]
    check(c)


def test_calls_of_all_sizes_one_behind_the_other():
    # blocks of 1 to 16 warps, which take tensor memory while blocks of the call before may still hold theirs
    lib()
    cs = [make(170, 3, 64, 8, [64] * 170, 64, seed=30, S=400), make(1, 1, 8, 8, [9], 128, seed=31),
          make(40, 3, 64, 8, [300] * 40, 32, seed=32, S=900), make(2, 2, 12, 2, [2000, 50], 64, seed=33),
          make(70, 1, 12, 2, [90] * 70, 128, seed=34, S=700), make(1, 4, 6, 1, [3], 32, seed=35)]
    want = [run(c)[0] for c in cs]
    names = ("q", "k_cache", "v_cache", "k_scales", "v_scales", "table", "lens")
    ds = [{x: c[x].cuda() for x in names} for c in cs]
    n = max(rsn.beam_attn_kv4_workspace(c["table"].shape[0], c["q_len"], c["q"].shape[1], c["k_cache"].shape[1],
                                        c["table"].shape[1]) for c in cs)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(d["q"]) for d in ds]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, d, o in zip(cs, ds, outs):
            rsn.beam_attn_kv4_fwd(o, d["q"], d["k_cache"], d["v_cache"], d["k_scales"], d["v_scales"], d["table"],
                                  d["lens"], ws, group=c["group"])
    torch.cuda.synchronize()
    assert all(torch.equal(o.cpu(), w) for o, w in zip(outs, want))


def test_two_streams_at_once():
    # calls that run side by side, each with its own workspace and output
    lib()
    cs = [make(4, 1, 12, 2, [700, 3, 90, 4000], 32, seed=21 + i) for i in range(2)]
    want = [run(c)[0] for c in cs]
    ds = [{x: c[x].cuda() for x in ("q", "k_cache", "v_cache", "k_scales", "v_scales", "table", "lens")} for c in cs]
    ws = [torch.empty(rsn.beam_attn_kv4_workspace(4, 1, 12, 2, 4000), dtype=torch.uint8, device="cuda") for _ in cs]
    outs = [torch.zeros_like(d["q"]) for d in ds]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, d, w, o in zip(streams, ds, ws, outs):
            rsn.beam_attn_kv4_fwd(o, d["q"], d["k_cache"], d["v_cache"], d["k_scales"], d["v_scales"], d["table"],
                                  d["lens"], w, group=32, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o.cpu(), w) for o, w in zip(outs, want))


def test_write_then_read():
    # the step as a server runs it: the new tokens' rows go in, and attention sees them
    lib()
    B, q_len, n_q, n_kv, group = 3, 2, 12, 2, 64
    c = make(B, q_len, n_q, n_kv, [2, 60, 129], group, seed=17)
    d = {x: c[x].cuda() for x in ("k_cache", "v_cache", "k_scales", "v_scales", "table", "lens")}
    k, v = (torch.randn((B * q_len, n_kv, D)).bfloat16() for _ in range(2))
    slots = torch.cat([c["table"][b, int(n) - q_len:int(n)] for b, n in enumerate(c["lens"])])
    rsn.beam_kv4_write_fwd(d["k_cache"], d["v_cache"], d["k_scales"], d["v_scales"], k.cuda(), v.cuda(),
                           slots.cuda(), group=group)
    for x, i in (("k", k), ("v", v)):
        c[x + "_cache"][slots], c[x + "_scales"][slots] = ref.kv4_write(i, group)
    check(c, d=d)
