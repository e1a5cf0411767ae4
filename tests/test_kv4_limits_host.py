"""CPU checks of the 4-bit paged cache at the ends of its ranges: what the C ABI refuses there, and
what q's three parts hold."""
import numpy as np
import pytest

import gated_deltanet_token_amd as gdn
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
