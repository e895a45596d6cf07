"""4-bit matrix-vector products against a plain 64-bit computation (needs a GB300).  The bound counts
half a step of BF16 for the output and FP32 sums of the exact products."""
import pytest
import torch

import residual_stream_norm_gb300 as rsn
from tests import _decode_ref as ref
from tests._gpu import CANARY, Guarded, lib

pytestmark = pytest.mark.gpu


def make(T, N, K, group, zeros, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, K), generator=g).bfloat16()
    w = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    s = (torch.randn((N, K // group), generator=g) * 0.01).bfloat16()
    z = torch.randint(0, 16, (N, K // group), generator=g, dtype=torch.uint8) if zeros else None
    return x, w, s, z


def check(x, w, s, z, group, y=None):
    T, N = x.shape[0], w.shape[0]
    out = Guarded((T, N)) if y is None else y
    xd = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda").copy_(x)
    rsn.beam_w4_matvec_fwd(out.view, xd, w.cuda(), s.cuda(), None if z is None else z.cuda(),
                           group=group)
    torch.cuda.synchronize()
    out.check()
    want, tol = ref.w4_matvec(x, w, s, z, group)
    d = (out.view.cpu().double() - want).abs()
    assert bool((d <= tol).all()), f"worst {float((d - tol).max()):.3g} past the bound"
    return out.view.cpu()


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("T,N,K,group", [
    (1, 1, 32, 32), (5, 70, 2560, 32), (20, 140, 4096, 64), (40, 130, 2048, 128), (3, 65, 6144, 128), (1, 5, 64, 64), (1, 16, 128, 128), (1, 17, 160, 32), (2, 33, 320, 64),
    (3, 100, 640, 128), (7, 31, 1056, 32), (8, 64, 4096, 128), (9, 65, 576, 64),
    (15, 40, 384, 128), (16, 257, 96, 32), (17, 16, 2048, 64), (31, 50, 1024, 128),
    (32, 48, 480, 32), (33, 90, 704, 64), (64, 130, 256, 128), (65, 24, 512, 32),
    (200, 70, 384, 128)])
def test_sizes(T, N, K, group, zeros):
    lib()
    check(*make(T, N, K, group, zeros, seed=T + N), group)


def test_beam_projections():
    lib()
    for T, N, K, group in ((1, 5120, 6144, 128), (4, 14336, 5120, 64)):
        check(*make(T, N, K, group, True, seed=N), group)


def test_one_weight_at_a_time():
    # every column's weight reaches its own product: x picks single columns
    lib()
    K, group = 256, 64
    _, w, s, z = make(1, 20, K, group, True, seed=3)
    for k0 in range(0, K, 32):
        x = torch.zeros((32, K), dtype=torch.bfloat16)
        x[torch.arange(32), k0 + torch.arange(32)] = 1.0
        check(x, w, s, z, group)


def test_strided_rows():
    lib()
    x, w, s, z = make(5, 37, 256, 128, True, seed=4)
    plain = check(x, w, s, z, 128)
    wide = torch.randn((5, 320)).bfloat16()
    wide[:, 8:264] = x
    y = Guarded((5, 64))
    full = y.view
    y.view = full[:, 3:40]
    assert torch.equal(check(wide[:, 8:264], w, s, z, 128, y=y), plain)
    assert bool((full[:, :3] == CANARY).all()) and bool((full[:, 40:] == CANARY).all())


def test_same_bits_every_time():
    lib()
    c = make(6, 500, 1024, 32, True, seed=5)
    first = check(*c, 32)
    assert all(torch.equal(first, check(*c, 32)) for _ in range(3))


def test_rows_do_not_mix():
    # a token's result does not depend on the other tokens, whatever they hold
    lib()
    x, w, s, z = make(9, 40, 256, 64, False, seed=6)
    plain = check(x, w, s, z, 64)
    x[4] = float("nan")
    x[7] = float("inf")
    y = Guarded((9, 40))
    rsn.beam_w4_matvec_fwd(y.view, x.cuda(), w.cuda(), s.cuda(), group=64)
    got = y.view.cpu()
    keep = [0, 1, 2, 3, 5, 6, 8]
    assert torch.equal(got[keep], plain[keep]) and bool(torch.isnan(got[4]).all())


def test_no_tokens():
    lib()
    _, w, s, _ = make(1, 8, 64, 32, False)
    rsn.beam_w4_matvec_fwd(torch.empty((0, 8), dtype=torch.bfloat16, device="cuda"),
                           torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), w.cuda(),
                           s.cuda(), group=32)
    torch.cuda.synchronize()


# 10 to 44 steps of 256 columns shared out over clusters of 1, 2, 4 and 8 blocks, so that shares start on
# every step of a window of 1024 columns
@pytest.mark.parametrize("T", [1, 8, 16])
@pytest.mark.parametrize("N,K,group,zeros", [
    (5120, 6144, 128, False), (14336, 5120, 64, True), (3584, 5120, 64, True),
    (7000, 5632, 32, True), (29000, 2560, 32, True), (130, 11264, 64, False)])
def test_windows_of_scales_from_memory(N, K, group, zeros, T):
    # Scales and zeros that differ from window to window: those of another window give another
    # result.  Everything is read from memory, which a buffer larger than the L2 cache sees to.
    lib()
    x, w, s, z = make(T, N, K, group, zeros, seed=N + T)
    window = torch.arange(K // group) * group // 1024
    s = (s.float() * 2.0 ** (window % 5 * 2 - 4)[None]).bfloat16()
    if zeros:
        z = ((z + 5 * window[None]) % 16).to(torch.uint8)
    want, tol = ref.w4_matvec(x, w, s, z, group)
    xd, wd, sd = x.cuda(), w.cuda(), s.cuda()
    zd = None if z is None else z.cuda()
    flush = torch.empty(2 ** 28, dtype=torch.uint8, device="cuda")
    first = None
    for i in range(6):
        y = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        flush.fill_(i)
        rsn.beam_w4_matvec_fwd(y, xd, wd, sd, zd, group=group)
        if first is None:
            first = y
            d = (y.cpu().double() - want).abs()
            assert bool((d <= tol).all()), f"worst {float((d - tol).max()):.3g} past the bound"
        assert torch.equal(y, first)
