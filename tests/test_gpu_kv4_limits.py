"""GPU checks of the 4-bit paged cache's calls at the ends of their ranges, with the bounds of
test_gpu_kv4_attention.py unless a test says otherwise."""
import numpy as np
import pytest
import torch

import gated_deltanet_token_amd as gdn
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


def guarded(shape, dtype, fill, rows=64):
    """(a buffer of `fill`, its middle of that shape)"""
    whole = torch.full((shape[0] + 2 * rows, *shape[1:]), fill, dtype=dtype, device="cuda")
    return whole, whole[rows:rows + shape[0]]


def untouched(whole, fill, rows=64):
    return bool((whole[:rows] == fill).all() and (whole[-rows:] == fill).all())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,qsl", [
    ([(50, 10), (60, 10), (70, 10)], [0, 25, 12, 900]), ([(50, 10), (60, 10), (70, 10)], [-9, 40, -3, 2 ** 31 - 1]),
    ([(300, 70), (400, 60), (90, 20)], [0, 140, 20, 2 ** 31 - 1]), ([(9000, 1), (5000, 1), (70, 1), (3, 0)], [0, 3, -2 ** 31, 2, 3000]),
    ([(9000, 2), (6000, 40), (70, 3)], [44, 10, 45, 0])], ids=["rows", "signs", "prompts", "decode", "parts"])
def test_malformed_query_start_loc_writes_nowhere_else(d, lens, qsl):
    """Bounds that decrease or lie outside: whose rows are whose is not said, but o's neighbours and the workspace's
    are as they were."""
    c = Case(63, lens, 8, 2, d, 16)
    T, c.qsl = c.q.shape[0], np.array(qsl, np.int32)
    n = gdn.gdn_paged_attention_kv4_workspace_size(T, len(lens), 8, 2, d, c.longest())
    whole, o = guarded(c.q.shape, torch.bfloat16, 77.0)
    ws_whole, ws = guarded((max(n, 1),), torch.uint8, 91, 4096)
    assert ws.data_ptr() % 256 == 0
    gdn.gdn_paged_attention_kv4(c.q, o=o, max_seq_len=c.longest(), scale=c.scale, workspace=ws, **c.gpu())
    torch.cuda.synchronize()
    assert untouched(whole, 77.0) and untouched(ws_whole, 91, 4096)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("loc", [[0, 50, 20, 900], [-7, 60, -2 ** 31, 2 ** 31 - 1], [90, 10, 100, 0]])
def test_malformed_out_start_loc_writes_nowhere_else(d, loc):
    c = Case(64, [(80, 1), (60, 1), (200, 1)], 2, 2, d, 16)
    g = c.gpu()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")                      # noqa: E731
    for starts in (None, i32([5, -3, 2 ** 31 - 1])):
        for which in ("kv", "k", "v"):
            outs = [guarded((100, 2, d), torch.bfloat16, 77.0) for _ in range(2)]
            gdn.gdn_paged_read_kv4(*(g[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale", "block_table")), starts, i32(loc),
                                   *(o if n in which else None for n, (_, o) in zip("kv", outs)))
            torch.cuda.synchronize()
            for n, (whole, o) in zip("kv", outs):
                assert untouched(whole, 77.0) and (n in which or (o == 77.0).all())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 3, 40], ids=["decode", "small", "large"])
@pytest.mark.parametrize("exponent", [-90, -100])
def test_light_keys_of_tiny_values_beside_heavy_ones_that_come_late(d, new, exponent):
    """Keys of 2^-17.17 of the heaviest's weight, with a value scale of 1.5 times 2^-100: their product is above 2^-117.
    It is rounded to bf16 once, as a normal number, also where the maximum is set behind the first keys.  (Sums below
    2^-126 are subnormal: a step of 2^-149 per sum, 700 of them.)"""
    c = Case(65, [(700, new)], 2, 1, d, 16, spread=0.0)
    c.q[:, :, 0] = 17.0
    c.kq[:, :, :, 0] = 0
    c.ks[...] = 127
    c.scale = float(1.01 * np.log(2.0))
    c.vs[...] = 1.5 * 2.0 ** exponent
    for i, p in enumerate(c.table[0, :44]):
        c.vq[p, 0, :, :] = c.r.integers(1, 8, (16, d)) + 8 * c.r.integers(0, 2, (16, 1))
        if i >= 18:
            c.kq[p, 0, ::5, 0] = 2                # these weigh 2^17.17 times the others
            c.vq[p, 0, ::5] = 0
    assert c.split_error() == 0.0
    want, mag = c.want()
    got = ref.values(c.run())
    heaviest = 1 / 140                            # at least, of the sum of weights
    bound = np.abs(want) * 2.0 ** -8 + mag * (2.0 ** -8 + 2.0 ** -11) + 700 * 2.0 ** -149 * 2.0 ** 8 * heaviest
    assert (np.abs(got - want) <= bound).all(), (np.abs(got - want) / bound).max()
