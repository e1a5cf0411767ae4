"""GPU checks of gdn_paged_attention_kv8 where the keys of prompt chunks are
divided over workgroups and joined: every head size, masks that leave some
parts without keys, bad codes in one part, small requests divided beside large
ones, and groups of more query heads than a small request has rows.

Bounds as in test_gpu_serving_attention (joining is fp32 arithmetic, covered
there).  Every call gets a workspace filled with NaN patterns, so that a part
that nobody wrote cannot pass as one."""
import numpy as np
import pytest
import torch

import gated_deltanet_token_amd as gdn
import serving_ref as ref
from test_gpu_serving_attention import Case, near

pytestmark = pytest.mark.gpu


def want(c, causal=True, window=0):
    """As serving_ref.attention, a request and kv head at a time."""
    q, (T, HQ, D), HK, page = ref.values(c.q), c.q.shape, c.kq.shape[1], c.kq.shape[2]
    G = HQ // HK
    o, mag = np.full((T, HQ, D), np.nan), np.full((T, HQ, D), -1.0)
    for s, L in enumerate(c.seq.tolist()):
        a, b = c.qsl[s], c.qsl[s + 1]
        if a == b:
            continue
        j, pos = np.arange(L), np.arange(L - (b - a), L)[:, None]
        ids = c.table[s][j // page]
        see = np.broadcast_to((ids >= 0) & (ids < c.kq.shape[0]), (b - a, L))
        if causal:
            see = see & (j <= pos)
        if window:
            see = see & (j > pos - window)
        at = np.where((ids >= 0) & (ids < c.kq.shape[0]), ids, 0)
        for h in range(HK):
            K = c.kq[at, h, j % page] * c.ks[at, h].astype(np.float64)[:, None]
            V = c.vq[at, h, :, j % page] * c.vs[at, h].astype(np.float64)[:, None]
            bad = np.isnan(V)
            for g in range(h * G, h * G + G):
                x = np.where(see, c.scale * (q[a:b, g] @ K.T), -np.inf)
                some = see.any(1)
                w = np.exp(x - np.where(some, x.max(1, initial=-np.inf), 0.0)[:, None])
                w /= np.where(some, w.sum(1), 1.0)[:, None]
                o[a:b, g], mag[a:b, g] = w @ np.where(bad, 0.0, V), w @ np.abs(np.where(bad, 0.0, V))
                o[a:b, g][(see.astype(np.float64) @ bad) > 0] = np.nan
    return o, mag


def workspace(c, longest):
    (T, hq, d), hk = c.q.shape, c.kq.shape[1]
    n = gdn.gdn_paged_attention_kv8_workspace_size(T, len(c.seq), hq, hk, d, longest)
    return torch.full((max(n, 1),), 255, dtype=torch.uint8, device="cuda")


def parts(c, longest):
    """How many parts a row's keys have at most, where only the large requests' are divided."""
    T, hq, d = c.q.shape
    return workspace(c, longest).numel() // (4 * T * hq * (d + 2))


def check(c, longest=None, **kw):
    longest = longest or c.longest()
    o = c.run(longest, workspace=workspace(c, longest), **kw)
    near(o, *want(c, **kw))
    return o


def test_the_reference_is_the_other_one():
    c = Case(1, [(70, 1), (90, 40), (33, 33)], 4, 2, 64, 16)
    c.vq[c.table[1, 3], 0, 5, 7], c.kq[c.table[2, 1], 1, 2, 3] = np.nan, np.nan
    c.table[0, 2] = -1
    for kw in (dict(), dict(causal=False), dict(window=20), dict(causal=False, window=5)):
        for a, b in zip(want(c, **kw), c.want(**kw)):
            np.testing.assert_allclose(a[np.isfinite(b)], b[np.isfinite(b)], rtol=1e-9, atol=1e-12)
        assert np.array_equal(np.isnan(want(c, **kw)[0]), np.isnan(c.want(**kw)[0]))


@pytest.mark.parametrize("d,page", [(64, 16), (128, 32), (256, 16), (256, 64)])
@pytest.mark.parametrize("lens,least", [([(640, 40)], 2), ([(1300, 300)], 4), ([(5000, 64)], 10), ([(3000, 100), (700, 50), (40, 40)], 6)])
def test_prompt_chunks(d, page, lens, least):
    c = Case(d + page, lens, 4, 2, d, page, spread=2.0)
    assert parts(c, c.longest()) >= least
    for kw in (dict(), dict(causal=False), dict(window=50), dict(window=700), dict(causal=False, window=300)):
        check(c, **kw)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_bounds_in_place_of_the_longest(d):
    c = Case(2, [(1900, 130), (300, 90)], 4, 2, d, 16)
    for longest in (600, 1024, 1899, 4000, 100000, 2 ** 31 - 1):
        assert parts(c, longest) >= 2
        check(c, longest)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_bad_codes_in_one_part(d):
    """NaN in a value and in a key that the later tokens see, in an early part, and where nobody looks."""
    for key in (200, 1100, 1250):
        c = Case(3, [(1300, 300)], 4, 2, d, 16)
        p, off = c.table[0, key // 16], key % 16
        c.vq[p, 0, 5, off] = np.nan
        c.kq[p, 1, off, 7] = np.nan
        o = ref.values(check(c))
        first = max(key - 1000, 0)
        assert np.isnan(o[first:, :2, 5]).all() and np.isnan(o[first:, 2:]).all()
        assert not np.isnan(o[:first]).any() and not np.isnan(o[first:, :2, 6]).any()
        check(c, window=1300 - key - 40)
    c = Case(4, [(1300, 300)], 4, 2, d, 16)
    for i in range(30):
        c.ks[c.table[0, i]], c.vs[c.table[0, i]] = np.nan, np.inf
        c.kq[c.table[0, i]], c.vq[c.table[0, i]] = np.nan, np.nan
    assert not np.isnan(ref.values(check(c, window=500))).any()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_missing_pages_in_parts(d):
    """Parts in which all pages, or all but one, are missing."""
    c = Case(5, [(1300, 70), (1000, 40)], 4, 2, d, 16)
    c.table[0, 16:40], c.table[0, 41:64] = -1, 10 ** 6
    c.table[1, :] = -1
    o = check(c)
    assert (o[70:] == 0).all() and (o[:70] != 0).any()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens", [[(5000, 1), (4100, 2), (3000, 60)], [(2500, 1)] * 3 + [(2500, 3), (5, 1), (9000, 33), (0, 0)]])
def test_small_requests_divided_beside_large_ones(d, lens):
    c = Case(d, lens, 4, 1, d, 16, spread=2.0)
    T = c.q.shape[0]
    small = 4 * len(lens) * 32 * (d + 2)                       # bytes a part of the small ones' rows
    assert workspace(c, c.longest()).numel() >= 4 * T * 4 * 2 * (d + 2) + 2 * small
    check(c)
    check(c, window=2000)


@pytest.mark.parametrize("hq,hk,d", [(40, 1, 64), (80, 2, 128), (40, 1, 256), (160, 1, 64), (160, 1, 128), (160, 1, 256)])
def test_groups_of_many_heads(hq, hk, d):
    """One token's rows alone are more than a small request has."""
    check(Case(hq, [(70, 1), (900, 1), (33, 1)], hq, hk, d, 16))
    c = Case(hq + 1, [(1200, 1), (300, 5), (40, 40), (17, 1), (0, 0)], hq, hk, d, 16)
    check(c)
    check(c, longest=10 ** 6)
    check(c, window=100)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_repeats_and_replays_are_bit_identical(d):
    c = Case(6, [(1300, 300), (2200, 1)], 4, 2, d, 16)
    first, g, ws, o = check(c), c.gpu(), workspace(c, 2200), torch.empty_like(c.q)

    def step():
        gdn.gdn_paged_attention_kv8(c.q, o=o, max_seq_len=2200, scale=c.scale, workspace=ws, **g)

    step()
    torch.cuda.synchronize()
    assert torch.equal(o, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        o.zero_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, first)
        torch.ones(1000, device="cuda").sum()               # eager work between the replays
