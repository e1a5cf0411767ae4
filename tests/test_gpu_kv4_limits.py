"""GPU checks of the 4-bit paged cache's calls at the ends of their ranges, with the bounds of
test_gpu_kv4_attention.py unless a test says otherwise."""
import numpy as np
import pytest

from test_gpu_kv4_attention import Case
from test_kv4_limits_host import largest_scale

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 3, 40], ids=["decode", "small", "large"])
def test_scores_of_zero_at_the_largest_scale(d, new):
    """q of zero: every key that is seen weighs the same, whatever the scale."""
    c = Case(60, [(300, new), (90, new)], 4, 2, d, 16, spread=0.0)
    for sign in (1, -1):
        c.scale = sign * float(largest_scale())
        c.check()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -149, -2.0 ** -140, 1e-38])
def test_large_products_at_a_scale_of_zero_and_tiny_ones(d, scale):
    """Products of q and k up to 2^126: at a scale of zero all keys weigh the same all the same."""
    c = Case(61, [(5, 1), (9, 3), (70, 40), (300, 1)], 4, 2, d, 16)
    c.q.mul_(2.0 ** 40)
    c.ks = np.where(c.ks == 255, 255, c.ks + 80).astype(np.uint8)
    c.scale = scale
    c.check()
