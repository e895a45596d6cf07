"""The mixture-of-experts layer at the ends of what its inputs may be, against the plain 64-bit computation (needs a
GB300)."""
import pytest
import torch

from tests._gpu import lib
from tests.test_gpu_moe_layer import check, make

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
