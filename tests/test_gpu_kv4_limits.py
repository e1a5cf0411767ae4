"""GPU checks of the 4-bit paged cache's calls at the ends of their ranges, with the bounds of
test_gpu_kv4_attention.py unless a test says otherwise."""
import numpy as np
import pytest
import torch

import serving_ref as ref
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


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 3, 40], ids=["decode", "small", "large"])
@pytest.mark.parametrize("top", [-109, -110, -111, -113, -117, -121, -124, -126])
def test_tiny_queries(d, new, top):
    """Two keys: one without score, and one that meets a single element of q, 2^-level of its block's
    largest of 2^top, with a score from -2.8 to -5.7: o = e^x / (1 + e^x) follows that element.
    Down to a largest of 2^-110 q's parts hold it exactly to level 7 and within 2^-15 of the largest
    from there on, below that within 2^-125."""
    S = 70
    c = Case(62, [(2, new)] * S, 1, 1, d, 16)
    r, at = c.r, c.table[:, 0]
    level = np.arange(S) % 10
    least = -126                                               # normal numbers
    level = np.minimum(level, top - least)
    small = (1 + r.integers(0, 128, S) / 128) * 2.0 ** (top - level)
    e = r.integers(1, 32, S) + 32 * r.integers(0, d // 32, S)
    q = np.zeros((S, d))
    q[:, ::32] = 1.9921875 * 2.0 ** top * r.choice([-1, 1], (S, d // 32))
    q[np.arange(S), e] = small
    c.q = torch.tensor(np.repeat(q, new, 0)[:, None], device="cuda").to(torch.bfloat16)
    assert np.array_equal(ref.values(c.q)[::new, 0], q)
    c.kq[...], c.vq[...], c.vs[...], c.scale = 0, 0, 1.0, 2.0 ** 6
    up = np.round(np.log2(4 / small)).astype(int) - 6
    assert (up <= 126).all()
    c.ks[at] = (127 + up)[:, None, None, None]
    c.kq[at, 0, 1, e] = 10                                     # -1
    c.vq[at, 0, 1] = 2                                         # 1
    x = -small * 2.0 ** up * c.scale
    want = np.repeat(np.exp(x) / (1 + np.exp(x)), new)
    off = np.where(level > 7, 2.0 ** -15 * 1.9921875 * 2.0 ** top, 0.0) if top >= -110 else 2.0 ** -125
    bound = want * (2 * 2.0 ** -8 + 2.0 ** -15 + np.repeat(np.expm1(off / small * np.abs(x)), new))
    err = np.abs(ref.values(c.run(causal=False))[:, 0] - want[:, None]).max(-1)
    assert (err <= bound).all(), (err / bound).max()
