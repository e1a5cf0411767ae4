"""CPU checks of the 4-bit paged cache at the ends of its ranges: what the C ABI refuses there, and
what q's three parts hold."""
import numpy as np
import pytest

import gated_deltanet_token_amd as gdn
import kv4_ref as kv4
from test_kv4_host import attn

INV = gdn.GDN_ERR_INVALID
# scores are in units of log2: the largest scale whose product with log2(e) is finite in fp32
LOG2E = np.float32(1.4426950408889634)


def largest_scale():
    x = np.float32(np.finfo(np.float32).max / np.float64(LOG2E))
    with np.errstate(over="ignore"):
        while np.isfinite(np.nextafter(x, np.float32(np.inf)) * LOG2E):
            x = np.nextafter(x, np.float32(np.inf))
        while not np.isfinite(x * LOG2E):
            x = np.nextafter(x, np.float32(0))
    return x


@pytest.mark.parametrize("sign", [1, -1])
def test_a_scale_whose_product_with_log2_e_is_infinite_is_refused(sign):
    """A score of zero times an infinite factor would be NaN."""
    x = largest_scale()
    assert 2.0 ** 127.4 < x < 2.0 ** 127.5
    for scale in (np.nextafter(x, np.float32(np.inf)), np.float32(3e38), np.finfo(np.float32).max):
        assert attn(scale=sign * float(scale)) == INV
        assert b"scale" in gdn.lib.gdn_last_error()
    # (this one is not: the call then stops at its next error, a missing o)
    assert attn(scale=sign * float(x), o=None) == INV and b"scale" not in gdn.lib.gdn_last_error()


def test_parts_of_q_at_the_end_of_their_range():
    """A block's power of two is 2^-111 at least, and the last part's step 2^-124: from a largest
    magnitude of 2^-110 on elements are held as for any other, below it within 2^-125."""
    sig = 1 + np.arange(128) / 128
    for top_exponent in range(-133, -104):
        for top in (1.0, 1.25, 1.9921875):
            top = top * 2.0 ** top_exponent
            for level in range(12):
                x = np.zeros((128, 32))
                x[:, 3], x[:, 7] = top, np.minimum(sig * 2.0 ** (top_exponent - level), top)
                err = np.abs(kv4.split(x) - x).max()
                at_most = 2.0 ** -125 if top_exponent < -110 else 0.0 if level <= 7 else 2.0 ** -15 * top
                assert err <= at_most, (top, level)
    # and below that the first statement does not hold
    x = np.zeros((1, 32))
    x[0, 3], x[0, 7] = 2.0 ** -111, 1.9921875 * 2.0 ** -118
    assert np.abs(kv4.split(x) - x).max() > 0
