"""The mixture-of-experts layer at the ends of what its inputs may be, against the plain 64-bit computation (needs a
GB300)."""
import pytest
import torch

import residual_stream_norm_gb300 as rsn
from tests._gpu import lib
from tests.test_gpu_moe_layer import check, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [5, 24])
def test_largest_tokens_with_the_smallest_weights(T):
    # |x| up to 2^127 beside weights that keep |x| |w| far below the documented 2^113
    lib()
    H = 256
    c = make(T, H, 24, seed=T)
    for e in (118, 122):
        big = {**c, "x": (c["x"].double() * 2.0 ** e).bfloat16(), "rw": (c["rw"].double() * 2.0 ** -e).float(),
               "w13": (c["w13"].double() * 2.0 ** -e).bfloat16()}
        big["x"][torch.arange(T), torch.arange(T) * 7 % H] = 2.0 ** (e + 5)
        check(big)


# up to 16 tokens are routed by every block of the first kernel, more by a kernel of its own; both list their experts' pairs
# in another way

@pytest.mark.parametrize("T", [1, 5, 16, 17, 40])
def test_ties_of_logits(T):
    # pairs of experts whose rows differ in one last bit, or not at all: the fast scores cannot tell, the exact sums do
    lib()
    c = make(T, 512, 8, seed=T)
    c["rb"].zero_()
    for e in range(0, 256, 2):
        c["rw"][e + 1] = c["rw"][e]
        if e % 4:
            i = e % 512
            c["rw"][e + 1, i] = torch.nextafter(c["rw"][e, i], torch.tensor(9.0))
    check(c)


@pytest.mark.parametrize("T", [16, 17, 40])
def test_all_scores_equal(T):
    lib()
    c = make(T, 64, 16, seed=T)
    c["rb"].zero_()
    c["rw"][:] = c["rw"][:1]
    check(c)


@pytest.mark.parametrize("first,local", [(0, 256), (0, 8), (100, 50)])
@pytest.mark.parametrize("T", [9, 16, 17, 40])
def test_tokens_without_a_number_do_not_mix(T, first, local):
    # tokens that hold NaN or infinities come to some experts too, and take places in their lists
    lib()
    c = make(T, 128, 40, first, local, seed=T)
    plain, ids, w = run(c)
    bad = [1, 4, T - 2]
    c["x"][bad[0], 3] = float("nan")
    c["x"][bad[1]] = float("inf")
    c["x"][bad[2], 100] = -float("inf")
    got, gids, gw = run(c)
    keep = [t for t in range(T) if t not in bad]
    for a, b in ((got, plain), (gids, ids), (gw, w)):
        assert torch.equal(a[keep], b[keep])
    assert bool((gids >= 0).all()) and bool((gids < 256).all())
    again = run(c)
    assert torch.equal(torch.nan_to_num(again[0], nan=7.0), torch.nan_to_num(got, nan=7.0)) and torch.equal(again[1], gids)


@pytest.mark.parametrize("T", [5, 20])
def test_activations_past_the_range_of_bf16(T):
    lib()
    c = make(T, 128, 40, seed=T)
    plain, _, _ = run(c)
    c["x"][2] = (c["x"][2].float() * 2.0 ** 70).bfloat16()
    got, _, _ = run(c)
    assert torch.equal(got[[0, 1] + list(range(3, T))], plain[[0, 1] + list(range(3, T))])
    assert bool(torch.isnan(got[2]).all())


def test_first_experts_that_the_c_type_cannot_hold():
    lib()
    c = make(3, 64, 16, 0, 8, seed=1)
    for first in (1 << 32, (1 << 32) + 5, -(1 << 32), 1 << 64):
        with pytest.raises(rsn.BeamError):
            run({**c, "first": first})
