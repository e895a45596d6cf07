"""Attention over the 4-bit cache at the ends of what a cache and a query may hold, against the plain 64-bit computation
(needs a GB300)."""
import pytest
import torch

from tests._gpu import lib
from tests.test_gpu_kv4 import check, make, run

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
