"""GPU checks of the 4-bit paged cache's calls at the ends of their ranges, with the bounds of
test_gpu_kv4_attention.py unless a test says otherwise."""
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
