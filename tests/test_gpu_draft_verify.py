"""Verification of drafted tokens against the same computation in whole numbers: equal in every token
(needs a GB300)."""
import numpy as np
import pytest
import torch

import residual_stream_norm_gb300 as rsn
from tests import _draft_ref as ref
from tests._gpu import lib

pytestmark = pytest.mark.gpu


def make(B, k, V, kind=torch.float32, draft=True, seed=0, sharp=2.0):
    g = torch.Generator().manual_seed(seed)
    logits = sharp * torch.randn((B, k + 1, V), generator=g)
    q = torch.softmax(logits[:, :k], 2).to(kind)
    p = torch.softmax(logits + 0.7 * torch.randn((B, k + 1, V), generator=g), 2).to(kind)
    tokens = torch.multinomial(q.float().view(B * k, V) + 1e-9, 1, generator=g).view(B, k) if k else \
        torch.empty((B, 0), dtype=torch.int64)
    if not draft:
        tokens = torch.where(torch.rand((B, k), generator=g) < 0.5, p[:, :k].argmax(2), tokens) if k else tokens
    return dict(tokens=tokens, target=p, draft=q if draft else None,
                u_accept=torch.rand((B, k), generator=g), u_sample=torch.rand(B, generator=g))


def run(c, lens=None, target=None, draft=None):
    B, k = c["tokens"].shape
    out = torch.full((B + 2, k + 1), 99, dtype=torch.int64, device="cuda")
    acc = torch.full((B + 2,), 99, dtype=torch.int32, device="cuda")
    draft = (None if c["draft"] is None else c["draft"].cuda()) if draft is None else draft
    rsn.beam_draft_verify_fwd(out[1:B + 1], acc[1:B + 1], c["tokens"].cuda(),
                              c["target"].cuda() if target is None else target, draft, c["u_accept"].cuda(),
                              c["u_sample"].cuda(),
                              None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    for t in (out, acc):
        assert bool((t[0] == 99).all()) and bool((t[-1] == 99).all())
    return out[1:B + 1].cpu().numpy(), acc[1:B + 1].cpu().numpy()


def check(c, lens=None, **kw):
    got = run(c, lens, **kw)
    want = ref.verify(c["tokens"], c["target"], c["draft"], c["u_accept"], c["u_sample"], lens)
    assert (got[1] == want[1]).all(), (got[1], want[1])
    assert (got[0] == want[0]).all(), (got[0], want[0])
    return got


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("B,k,V", [(1, 1, 1), (1, 0, 10), (2, 3, 2), (3, 4, 33), (5, 7, 1000), (1, 4, 2047),
                                   (4, 2, 2049), (2, 5, 16384), (3, 1, 50021), (40, 3, 129)])
def test_sizes(B, k, V, draft, kind):
    lib()
    check(make(B, k, V, kind, draft, seed=B + V))


def test_large_vocabularies():
    lib()
    for V in (160_000, (1 << 20) - 1):
        check(make(2, 2, V, seed=V, sharp=3.0))


@pytest.mark.parametrize("V", [300, 40_000, 70_000])
def test_more_blocks_than_have_room_at_a_time(V):
    lib()
    check(make(160, 1, V, seed=V, sharp=3.0))


def test_more_tokens_than_a_warp_has_lanes():
    # all accepted, or the first refusal at each place around a warp's end
    lib()
    B, k, V = 6, 70, 40
    c = make(B, k, V, seed=1)
    c["u_accept"].fill_(0.0)
    for b, i in enumerate((0, 31, 32, 33, 69)):
        c["u_accept"][b, i] = 0.999
        c["draft"][b, i, c["tokens"][b, i]] = 1.0
        c["target"][b, i, c["tokens"][b, i]] = 1e-3
    got = check(c)
    assert got[1].tolist() == [0, 31, 32, 33, 69, 70]


def test_lengths_of_drafts():
    lib()
    c = make(6, 5, 300, seed=2)
    check(c, [0, 1, 3, 5, -2, 9])
    c["u_accept"].fill_(0.0)
    assert check(c, [0, 1, 3, 5, -2, 9])[1].tolist() == [0, 1, 3, 5, 0, 5]


def test_random_numbers_at_their_ends():
    lib()
    c = make(8, 2, 500, seed=3)
    c["u_sample"] = torch.tensor([0.0, 2.0 ** -60, 0.99999994, 1.0, 7.0, -1.0, float("nan"), 2.0 ** -149])
    c["u_accept"][:, 0] = torch.tensor([0.0, 1.0, 0.99999994, float("nan"), 2.0, -1.0, 0.5, float("inf")])
    check(c)
    # the last token, and the first of weight, are reached
    c["target"].zero_()
    c["target"][:, :, 499] = 1.0
    c["target"][:, :, 17] = 2.0 ** -43
    check(c)


def test_nothing_left_to_draw_from():
    # equal distributions that were refused all the same: the target's own; zeros everywhere: -1
    lib()
    c = make(4, 1, 200, seed=4)
    c["draft"] = c["target"][:, :1].clone()
    c["u_accept"].fill_(1.0)
    assert (check(c)[1] == 0).all()
    c["target"][2:] = 0
    got = check(c)
    assert (got[0][2:, 0] == -1).all()
    c["draft"] = None
    c["target"][0] = 0
    c["target"][0, :, c["tokens"][0, 0]] = 1e-12
    check(c)


def test_probabilities_that_are_none():
    lib()
    c = make(5, 2, 700, seed=5)
    nan, inf = float("nan"), float("inf")
    c["target"][0, :, 5] = nan
    c["target"][1, :, 6] = inf
    c["target"][2, :, 7] = -1.0
    c["draft"][3, :, 8] = nan
    c["draft"][4, :, 9] = inf
    c["tokens"][0, 0], c["tokens"][3, 0], c["tokens"][1, 0] = 5, 8, 6
    check(c)


def test_tokens_outside_the_vocabulary():
    lib()
    for draft in (True, False):
        c = make(3, 2, 64, seed=6, draft=draft)
        c["u_accept"].fill_(0.0)
        c["tokens"][0, 0], c["tokens"][1, 1], c["tokens"][2, 0] = -1, 64, 1 << 40
        got = check(c)
        assert got[1][0] == 0 and got[1][2] == 0


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_strides_and_alignments(kind):
    lib()
    B, k, V = 3, 2, 1001
    c = make(B, k, V, kind, seed=7)
    wide = torch.zeros((k + 1, B, V + 9), dtype=kind, device="cuda")
    other = torch.zeros((B, k + 2, V + 3), dtype=kind, device="cuda")
    for off in (0, 1, 5):
        wide[:, :, off:off + V] = c["target"].cuda().transpose(0, 1)
        other[:, 1:k + 1, 2:2 + V] = c["draft"].cuda()
        check(c, target=wide[:, :, off:off + V].transpose(0, 1), draft=other[:, 1:k + 1, 2:2 + V])
    # one distribution for all positions
    c["draft"] = c["draft"][:, :1].expand(B, k, V)
    check(c, draft=c["draft"][:, :1].cuda().expand(B, k, V))


def test_distribution_is_the_target():
    # over an even grid of random numbers the drawn tokens come as often as the target says
    lib()
    n, V = 4096, 37
    g = torch.Generator().manual_seed(8)
    p, q = (torch.softmax(1.5 * torch.randn(V, generator=g), 0) for _ in range(2))
    u = torch.rand((n, 64), generator=g)
    x = torch.multinomial(q, n * 64, replacement=True, generator=g).view(n * 64, 1)
    c = dict(tokens=x, target=torch.stack((p, p)).expand(n * 64, 2, V), draft=q.expand(n * 64, 1, V),
             u_accept=u.view(-1, 1), u_sample=torch.rand(n * 64, generator=g))
    out, _ = run(c, target=torch.stack((p, p)).cuda().expand(n * 64, 2, V), draft=q.cuda().expand(n * 64, 1, V))
    freq = np.bincount(out[:, 0], minlength=V) / (n * 64)
    # six standard deviations of a share of 2^18 draws
    assert (np.abs(freq - p.numpy()) <= 6 * np.sqrt(p.numpy() / (n * 64))).all()


def test_same_bits_in_a_graph():
    lib()
    c = make(4, 3, 5000, seed=9)
    want = check(c)
    d = {x: c[x].cuda() for x in c}
    out = torch.zeros((4, 4), dtype=torch.int64, device="cuda")
    acc = torch.zeros(4, dtype=torch.int32, device="cuda")

    def call():
        rsn.beam_draft_verify_fwd(out, acc, d["tokens"], d["target"], d["draft"], d["u_accept"], d["u_sample"])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert (out.cpu().numpy() == want[0]).all()


def test_no_sequences():
    lib()
    c = make(1, 2, 10, seed=1)
    c = {x: t[:0] for x, t in c.items()}
    assert run(c)[0].shape == (0, 3)
