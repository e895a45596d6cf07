"""Attention over the 4-bit cache at the ends of what a cache and a query may hold, against the plain 64-bit computation
(needs a GB300)."""
import pytest
import torch

from tests import _draft_ref as ref
from tests._gpu import lib
from tests.test_gpu_kv4 import check, check_write, make, run

pytestmark = pytest.mark.gpu
NAN = float("nan")


def scores(c, b, places, s):
    """Keys of sequence b: at `places` score s, elsewhere 0 (one KV head, a query of ones in column 0, sm_scale 1)."""
    at = c["table"][b]
    c["q"].zero_()
    c["q"][..., 0] = 1.0
    c["k_cache"][at] = 0
    c["k_scales"][at] = 0
    c["k_cache"][at[places], 0, 0] = 1
    c["k_scales"][at[places], 0, 0, 0] = s


@pytest.mark.parametrize("n", [5, 64, 100, 900, 9000])
@pytest.mark.parametrize("what", ["scale", "minimum"])
def test_a_seen_key_that_holds_nan_shows_whatever_its_weight(n, what):
    # weights far below what FP32 holds, in full tiles and in the last one, in parts that others outweigh
    lib()
    c = make(1, 1, 6, 1, [n], 128, seed=n)
    scores(c, 0, [n // 2], 300.0)
    clean, lse = run(c, sm_scale=1.0)
    assert bool(torch.isfinite(clean).all())
    for place in {0, 1, n // 2 - 1, n - 1}:
        d = {**c, "v_scales": c["v_scales"].clone()}
        d["v_scales"][c["table"][0, place], 0, 0, 0 if what == "scale" else 1] = NAN
        got, z = run(d, sm_scale=1.0)
        assert bool(torch.isnan(got).all()), place
        assert torch.equal(z, lse)


@pytest.mark.parametrize("n", [1000, 2000])
@pytest.mark.parametrize("group", [32, 128])
def test_scales_that_other_rows_see_do_not_cost_bits(n, group):
    # 24 query tokens behind a window: the first ones see 23 keys that the last does not, whose values' scales rise from
    # tile to tile (2^7 and 2^15 beside 1), and share tiles with keys that all see.  The last row's weights of all keys but
    # one are 2^-25, and that one's value is 0: what they add up to is all of the output.  The batch is so large that a
    # warp takes all of a sequence's tiles in turn.
    lib()
    B, q_len, n_sink, window = 1800, 24, 16, n - 50
    c = make(B, q_len, 1, 1, [n] * B, group, seed=n, S=n)
    c["table"][0] = torch.randperm(n, generator=torch.Generator().manual_seed(n))
    scores(c, 0, [n - 1 - window // 2], 17.34)
    at, lo = c["table"][0], n - q_len + 1 - window          # lo: first key behind the sinks that the first row sees
    c["v_scales"][at] = torch.tensor([1.0, 0.0]).bfloat16()
    c["v_scales"][at[lo:lo + 16], :, :, 0] = 2.0 ** 7
    c["v_scales"][at[lo + 16:lo + 23], :, :, 0] = 2.0 ** 15
    c["v_cache"][at[n - 1 - window // 2]] = 0
    out, _ = run(c, window, n_sink, sm_scale=1.0)
    (want, _), (tol, _) = ref.kv4_attention(c["q"][:q_len], c["k_cache"], c["v_cache"], c["k_scales"], c["v_scales"],
                                            c["table"][:1], c["lens"][:1], q_len, 1.0, window, n_sink)
    d = (out[:q_len].double() - want).abs()
    assert bool((d <= tol).all()), f"worst {float((d / tol).max()):.3g} of the bound"


@pytest.mark.parametrize("n", [1, 64, 3000])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_largest_scales_of_values(n, group):
    # one key with scales from 2^127 on, whose exponent is FP32's last, codes 0 and 1 beside a minimum of -2^126
    lib()
    c = make(1, 1, 6, 1, [n], group, seed=n + group)
    c["v_cache"] &= 0x11
    big = c["table"][0, n // 2]
    for far, score in ((2.0 ** 127 * 1.25, 30.0), (2.0 ** 127, 0.0)):
        scores(c, 0, [n // 2], score)
        c["v_scales"][..., 0], c["v_scales"][..., 1] = 1.0, 0.5
        c["v_scales"][big, ..., 0], c["v_scales"][big, ..., 1] = far, -(2.0 ** 126)
        check(c, sm_scale=1.0)


def test_largest_queries():
    # |q| |sm_scale| just below 2^117 beside keys so small that scores are ordinary; the other row has NaN from infinite ones
    lib()
    c = make(2, 2, 6, 1, [70, 150], 64, seed=1)
    c["q"] = (c["q"].float().clamp(-3.9, 3.9) * 2.0 ** 115).bfloat16()
    c["k_scales"] = (c["k_scales"].float() * 2.0 ** -118).bfloat16()
    clean, lse = check(c, sm_scale=0.5)
    c["q"][1, 2, 5] = float("inf")
    out, z = run(c, sm_scale=0.5)
    assert bool(torch.isnan(out[1, 2]).all()) and bool(torch.isnan(z[1, 2]))
    keep = torch.ones((4, 6), dtype=torch.bool)
    keep[1, 2] = False
    assert torch.equal(out[keep], clean[keep]) and torch.equal(z[keep], lse[keep])


@pytest.mark.parametrize("group", [32, 64, 128])
def test_write_of_any_bits(group):
    # all exponents in one group, and groups whose values are close to one another
    lib()
    g = torch.Generator().manual_seed(group)
    k = torch.randint(-1 << 15, 1 << 15, (150, 2, 128), generator=g, dtype=torch.int16)
    v = torch.randint(0, 1 << 15, (150, 2, 1), generator=g, dtype=torch.int16)
    v = v + torch.randint(0, 40, (150, 2, 128), generator=g, dtype=torch.int16)
    check_write(k.view(torch.bfloat16), v.view(torch.bfloat16), torch.randperm(200, generator=g)[:150], 200, group)
