"""GPU checks of gdn_paged_attention_kv8 for requests that are longer than
their block-table rows, up to the length 2^31 - 1 that gdn_build_step_tables
saturates at: what lies past the row is not seen, and a window past it leaves
the token without keys.  Bounds as in test_gpu_serving_attention."""
import numpy as np
import pytest

from test_gpu_serving_attention import Case

pytestmark = pytest.mark.gpu
TOP = 2 ** 31 - 1


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens", [[(100, 1), (70, 1), (50, 1)], [(100, 1), (90, 3), (200, 60), (40, 1)]], ids=["decode", "mixed"])
@pytest.mark.parametrize("window", [1, 100, 447, 5000])
@pytest.mark.parametrize("short", [0, 64, 500])
def test_windows_past_the_row(d, lens, window, short):
    c = Case(d + window, lens, 4, 2, d, 16)
    far = list(range(len(lens) - 1))                     # all but the last request
    c.seq[far] = TOP - short
    first_of_last = int(c.qsl[-2])
    for longest in (300, TOP):
        o = c.check(longest=longest, window=window)
        assert (o[:first_of_last] == 0).all() and (o[first_of_last:] != 0).any()


@pytest.mark.parametrize("d", [64, 256])
def test_saturated_lengths_see_their_row(d):
    c = Case(5, [(64, 1), (33, 2), (128, 70)], 4, 2, d, 16, spare_cols=0)
    c.seq[:] = TOP
    c.table = np.ascontiguousarray(c.table[:, :2])
    c.check(longest=300)
    c.check(longest=300, causal=False)
    o = c.check(longest=300, causal=False, window=9)
    assert (o == 0).all()


def test_a_window_that_reaches_back_into_the_row():
    """A request one token, and one page, longer than its row, with windows that end in it."""
    c = Case(6, [(200, 1), (200, 50), (70, 1)], 8, 2, 128, 16)
    c.table = np.ascontiguousarray(c.table[:, :12])       # 192 keys
    for window in (4, 8, 9, 20, 300):
        o = c.check(window=window)
        assert (o[0] == 0).all() == (window <= 8)
