"""The mixture-of-experts layer for a few tokens against a plain 64-bit computation (needs a GB300): the
choice of experts equal to the oracle's, the output within a bound that counts half a step of BF16 for the
activations and the result, and FP32 sums."""
import pytest
import torch

import residual_stream_norm_gb300 as rsn
from tests import _draft_ref as ref
from tests._gpu import Guarded, lib

pytestmark = pytest.mark.gpu


def make(T, H, F, first=0, local=256, seed=0):
    g = torch.Generator().manual_seed(seed)
    return dict(x=torch.randn((T, H), generator=g).bfloat16(),
                rw=torch.randn((256, H), generator=g) * H ** -0.5, rb=0.05 * torch.randn(256, generator=g),
                w13=(torch.randn((local, 2 * F, H), generator=g) * H ** -0.5).bfloat16(),
                w2=(torch.randn((local, H, F), generator=g) * F ** -0.5).bfloat16(), first=first)


def run(c, scaling=2.5, xd=None, out=None, outputs=True):
    T, H = c["x"].shape
    local, _, F = c["w2"].shape
    n = rsn.beam_moe_layer_workspace(T, H, F, local)
    ws = Guarded((max(16, n) // 4,), dtype=torch.float32)
    ws.view.fill_(float("nan"))
    out = out or Guarded((T, H))
    ids = torch.full((T, 8), -5, dtype=torch.int32, device="cuda") if outputs else None
    w = torch.full((T, 8), -5.0, device="cuda") if outputs else None
    dev = c.setdefault("dev", {x: c[x].cuda() for x in ("rw", "rb", "w13", "w2")})
    rsn.beam_moe_layer_fwd(out.view, c["x"].cuda() if xd is None else xd, dev["rw"], dev["rb"], dev["w13"],
                           dev["w2"], ws.view.view(torch.uint8), first_expert=c["first"],
                           routed_scaling=scaling, topk_ids_out=ids, topk_w_out=w)
    torch.cuda.synchronize()
    out.check()
    ws.check()
    return out.view.cpu(), ids if ids is None else ids.cpu(), w if w is None else w.cpu()


def check(c, scaling=2.5, **kw):
    out, ids, w = run(c, scaling, **kw)
    want_ids, want_w = ref.moe_route(c["x"], c["rw"], c["rb"])
    local = c["w2"].shape[0]
    if ids is not None:
        assert (ids.numpy() == want_ids).all()
        assert (w.numpy() == want_w).all()
    inside = lambda t: lambda e: t[e] if 0 <= e < local else None  # noqa: E731
    want, tol = ref.moe_layer(c["x"], want_ids, want_w, inside(c["w13"]), inside(c["w2"]), c["first"], scaling)
    d = (out.double() - want).abs()
    assert bool((d <= tol).all()), f"worst {float((d - tol).max()):.3g} past the bound"
    assert rsn.beam_device_faults() == 0
    return out


@pytest.mark.parametrize("T,H,F", [(1, 8, 8), (1, 64, 32), (2, 40, 8), (3, 512, 64), (5, 1032, 24), (8, 160, 136),
                                   (9, 256, 40), (17, 320, 72), (33, 96, 104), (64, 640, 320), (1, 5000, 16),
                                   (1, 16384, 8), (4, 24, 1000), (2, 16, 3000)])
def test_sizes(T, H, F):
    lib()
    check(make(T, H, F, seed=T + H))


@pytest.mark.parametrize("first,local", [(0, 32), (96, 32), (224, 32), (255, 1), (0, 1), (100, 7), (128, 128)])
def test_shares_of_experts(first, local):
    lib()
    check(make(20, 64, 48, first, local, seed=first))


def test_shares_add_up():
    lib()
    c = make(6, 128, 64, seed=3)
    whole, _, _ = run(c)
    parts = 0
    for first in range(0, 256, 64):
        p = {**c, "w13": c["w13"][first:first + 64], "w2": c["w2"][first:first + 64], "first": first}
        p.pop("dev", None)
        parts = parts + run(p)[0].double()
    # each part and the whole are off by half a step of BF16
    tol = 2.0 ** -8 * 6 * parts.abs().max()
    assert bool(((parts - whole.double()).abs() <= tol).all())


@pytest.mark.parametrize("T", [8, 9, 100, 256])
def test_all_tokens_to_the_same_experts(T):
    # the bias decides: experts 0-7 get every token, in passes of 8
    lib()
    c = make(T, 72, 24, seed=T)
    c["rb"][:8] += 50
    out, ids, _ = run(c)
    assert bool((ids.sort(1).values == torch.arange(8)).all())
    check(c)


def test_most_tokens():
    lib()
    check(make(256, 64, 24, seed=4))


def test_no_expert_here():
    lib()
    c = make(5, 64, 16, 200, 8, seed=5)
    c["rb"][200:208] = -100
    assert bool((run(c)[0] == 0).all())


def test_beam_shapes():
    # a few experts of Beam's tensor-parallel and expert-parallel shares
    lib()
    for H, F, first, local, T in ((5120, 320, 40, 12, 3), (5120, 2560, 8, 3, 10)):
        c = make(T, H, F, first, local, seed=F)
        c["rb"][first:first + local] += 2
        check(c)


def test_strided_rows():
    lib()
    c = make(7, 64, 32, seed=6)
    plain, _, _ = run(c)
    wide = torch.randn((7, 100)).bfloat16().cuda()
    wide = torch.cat((wide, wide[:, :4]), 1)
    wide[:, 16:80] = c["x"].cuda()
    out = Guarded((7, 104))
    full = out.view.fill_(3.0)
    out.view = full[:, 8:72]
    got, _, _ = run(c, xd=wide[:, 16:80], out=out)
    assert torch.equal(got, plain)
    assert bool((full[:, :8] == 3).all()) and bool((full[:, 72:] == 3).all())


def test_without_the_choice():
    lib()
    c = make(7, 64, 32, seed=7)
    assert torch.equal(run(c)[0], run(c, outputs=False)[0])


@pytest.mark.parametrize("scaling", [1.0, 0.0, -3.5])
def test_scaling(scaling):
    lib()
    check(make(3, 64, 32, seed=8), scaling)


def test_tokens_do_not_mix():
    lib()
    c = make(9, 128, 40, seed=9)
    plain, ids, _ = run(c)
    c["x"][4, 3] = float("nan")
    c["x"][6] = float("inf")
    got, gids, _ = run(c)
    keep = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(got[keep], plain[keep]) and torch.equal(gids[keep], ids[keep])
    assert bool(torch.isnan(got[4]).all())


def test_near_ties_of_logits():
    # two experts whose rows differ in one last bit, or not at all: the order is that of the exact sums
    lib()
    c = make(64, 512, 8, seed=10)
    c["rb"].zero_()
    for e in range(0, 256, 2):
        c["rw"][e + 1] = c["rw"][e]
        if e % 4:
            i = e % 512
            c["rw"][e + 1, i] = torch.nextafter(c["rw"][e, i], torch.tensor(9.0))
    check(c)


def test_same_bits_every_time_and_in_a_graph():
    lib()
    c = make(21, 256, 104, seed=11)
    first, ids, w = run(c)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(c), (first, ids, w)))
    x, d = c["x"].cuda(), c["dev"]
    ws = torch.empty(rsn.beam_moe_layer_workspace(21, 256, 104), dtype=torch.uint8, device="cuda")
    out = torch.zeros((21, 256), dtype=torch.bfloat16, device="cuda")

    def call():
        rsn.beam_moe_layer_fwd(out, x, d["rw"], d["rb"], d["w13"], d["w2"], ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        call()
    for _ in range(3):
        out.fill_(7)
        graph.replay()
        assert torch.equal(out.cpu(), first)


def test_two_streams_at_once():
    lib()
    cs = [make(T, 256, 104, seed=13 + T) for T in (5, 40)]
    want = [run(c)[0] for c in cs]
    xs = [c["x"].cuda() for c in cs]
    ws = [torch.empty(rsn.beam_moe_layer_workspace(len(x), 256, 104), dtype=torch.uint8, device="cuda") for x in xs]
    outs = [torch.zeros_like(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, c, x, w, o in zip(streams, cs, xs, ws, outs):
            d = c["dev"]
            rsn.beam_moe_layer_fwd(o, x, d["rw"], d["rb"], d["w13"], d["w2"], w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o.cpu(), w) for o, w in zip(outs, want))


@pytest.mark.parametrize("T,H,F", [(256, 16384, 8), (256, 8, 32768)])
def test_largest_sizes(T, H, F):
    lib()
    c = make(T, H, F, 40, 2, seed=T + F)
    c["rb"][40:42] += 50  # every token comes here
    check(c)


def test_no_tokens():
    lib()
    c = make(1, 64, 16, seed=12)
    c["x"] = c["x"][:0]
    assert run(c)[0].shape == (0, 64)
