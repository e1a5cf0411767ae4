"""CPU checks of what gdn_paged_attention_kv8 refuses because its kernels could
not address it."""
import pytest

import gated_deltanet_token_amd as gdn
from test_serving_host import UNS, P, attn


@pytest.mark.parametrize("heads,page,d", [(131072, 64, 256), (131073, 64, 256), (262144, 64, 128), (1 << 20, 32, 64), (2 ** 31 - 64, 16, 64)])
def test_pages_of_2_gib_are_refused(heads, page, d):
    """The prompt kernels' offsets within a page, of all kv heads, are 32-bit."""
    w = heads * d
    assert attn(HQ=heads, HK=heads, page=page, D=d, qs=w, os=w, T=1, S=1, n=1) == UNS
    assert b"2^31" in gdn.lib.gdn_last_error()


def test_a_page_just_below_that_is_not():
    """131,071 heads: refused for its o alone, which is q."""
    assert attn(HQ=131071, HK=131071, page=64, D=256, qs=131071 * 256, os=131071 * 256, T=1, S=1, n=1, o=P[0]) == gdn.GDN_ERR_INVALID
    assert b"o overlaps q" in gdn.lib.gdn_last_error()
