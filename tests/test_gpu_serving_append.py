"""GPU checks of gdn_rope_append_kv8 against the formulas in 64 bits.

Rotation and quantisation are formed in 64 bits on both sides and rounded the
same way, so codes and scales are compared for equality; q within half a bf16
step (2^-8 relative) and one fp32 step."""
import numpy as np
import pytest
import torch

import gated_deltanet_token_amd as gdn
import serving_ref as ref

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def bf(a):
    return torch.tensor(np.asarray(a, np.float32), device="cuda").to(torch.bfloat16)


def make_cache(r, pages, hk, page, d):
    """A cache with content, quantised the way the call does it."""
    kq, ks = ref.quantised(r.standard_normal((pages, hk, page, d)) * np.exp(r.standard_normal((pages, hk, 1, 1))))
    vq, vs = ref.quantised(r.standard_normal((pages, hk, page, d)) * np.exp(r.standard_normal((pages, hk, 1, 1))))
    f8 = lambda x: torch.tensor(x, dtype=torch.float32, device="cuda").to(F8)          # noqa: E731
    f32 = lambda x: torch.tensor(x, dtype=torch.float32, device="cuda")                # noqa: E731
    return [f8(kq), f8(vq.transpose(0, 1, 3, 2)).contiguous(), f32(ks), f32(vs)]


def as_ref(c):
    k, v, ks, vs = (ref.values(x) for x in c)
    return k, v.transpose(0, 1, 3, 2), ks, vs


def check(q, k, v, pos, slots, freq, cache, interleaved=False, rope_scale=1.0, q_out=None):
    k0, v0, ks0, vs0 = as_ref(cache)
    qr, kr, vr = (None if x is None else ref.values(x) for x in (q, k, v))
    if q is not None and q_out is None:
        q_out = torch.full((q.shape[0], q.shape[1], q.shape[2]), 99.0, dtype=torch.bfloat16, device="cuda")
    f = torch.tensor(freq, dtype=torch.float64, device="cuda") if len(freq) else None
    gdn.gdn_rope_append_kv8(q, k, v, torch.tensor(pos, dtype=torch.int32, device="cuda"),
                            torch.tensor(slots, dtype=torch.int64, device="cuda"), f, q_out, *cache, interleaved=interleaved,
                            rope_scale=rope_scale)
    torch.cuda.synchronize()
    krot = ref.rotate(kr, pos, freq, rope_scale, interleaved).astype(np.float32).astype(np.float64)
    want_k, want_ks = ref.append(krot, slots, k0, ks0)
    want_v, want_vs = ref.append(vr, slots, v0, vs0)
    got = as_ref(cache)
    for name, g, w in (("k_scale", got[2], want_ks), ("v_scale", got[3], want_vs), ("k", got[0], want_k), ("v", got[1], want_v)):
        assert np.array_equal(g, w, equal_nan=True), "%s: %d of %d differ" % (name, (g != w).sum(), g.size)
    if q is not None:
        want = ref.rotate(qr, pos, freq, rope_scale, interleaved)
        err = np.abs(ref.values(q_out) - want)
        assert (err <= np.abs(want) * (2.0 ** -8 + 2.0 ** -23) + 1e-38).all(), err.max()
    return q_out


def runs(r, spec, page, pages):
    """positions and slots of requests given as (context, new): pages at random ids."""
    ids = list(r.permutation(pages))
    pos, slots = [], []
    for c, n in spec:
        have = {}
        for p in range(c, c + n):
            if p // page not in have:
                have[p // page] = ids.pop()
            pos.append(p)
            slots.append(int(have[p // page]) * page + p % page)
    return pos, slots


MIX = [(0, 1), (5, 1), (15, 1), (16, 1), (63, 1), (0, 40), (7, 9), (31, 2), (60, 5), (12, 130), (3, 0), (64, 64)]


@pytest.mark.parametrize("d,page,rot,interleaved", [
    (64, 16, 64, False), (64, 32, 32, True), (64, 64, 0, False), (128, 16, 128, True), (128, 32, 64, False), (128, 64, 48, False),
    (128, 64, 128, False), (256, 16, 64, False), (256, 32, 256, True), (256, 64, 256, False), (256, 16, 16, True)])
@pytest.mark.parametrize("hq,hk", [(4, 2), (5, 5), (8, 1)])
def test_mixed_runs(d, page, rot, interleaved, hq, hk):
    r = np.random.default_rng(d + page + rot + hq)
    pos, slots = runs(r, MIX, page, 60)
    T = len(pos)
    qkv = bf(r.standard_normal((T, hq + 2 * hk, d)) * np.exp(r.standard_normal((T, hq + 2 * hk, 1))))
    check(qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], pos, slots, ref.frequencies(rot), make_cache(r, 60, hk, page, d),
          interleaved)


def test_q_in_place_in_the_projection():
    r = np.random.default_rng(1)
    pos, slots = runs(r, [(3, 20), (100, 1)], 16, 9)
    qkv = bf(r.standard_normal((21, 8, 128)))
    before = qkv.clone()
    for rot, il in ((128, True), (64, False), (32, True)):
        qkv.copy_(before)
        check(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], pos, slots, ref.frequencies(rot), make_cache(r, 9, 2, 16, 128), il, 1.25,
              q_out=qkv[:, :4])
        assert torch.equal(qkv[:, 4:], before[:, 4:]) and torch.equal(qkv[:, :4, rot:], before[:, :4, rot:])


def test_without_q():
    r = np.random.default_rng(2)
    pos, slots = runs(r, [(0, 33), (9, 1)], 32, 5)
    check(None, bf(r.standard_normal((34, 3, 64))), bf(r.standard_normal((34, 3, 64))), pos, slots, ref.frequencies(64),
          make_cache(r, 5, 3, 32, 64))


def test_many_tokens_take_the_wider_q_blocks():
    r = np.random.default_rng(3)
    pos, slots = runs(r, [(0, 1500), (777, 31)], 16, 100)
    check(bf(r.standard_normal((1531, 3, 64))), bf(r.standard_normal((1531, 1, 64))), bf(r.standard_normal((1531, 1, 64))), pos,
          slots, ref.frequencies(64), make_cache(r, 100, 1, 16, 64), True)


def test_far_positions_scaled():
    r = np.random.default_rng(4)
    f, m = gdn.gdn_rope_frequencies(128, 1e6, "yarn", 32.0, original_context=32768)
    pos = [0, 1, 1048575, 999983, 2 ** 31 - 1]
    slots = [16 * i for i in range(5)]
    check(bf(r.standard_normal((5, 2, 128))), bf(r.standard_normal((5, 1, 128))), bf(r.standard_normal((5, 1, 128))), pos, slots, f,
          make_cache(r, 5, 1, 16, 128), rope_scale=m)


@pytest.mark.parametrize("page", [16, 64])
def test_scale_grows_token_by_token(page):
    """Decode steps into the same pages with ever larger, then smaller, tokens."""
    r = np.random.default_rng(5)
    cache = make_cache(r, 4, 2, page, 64)
    for i in range(page + 5):
        p = i
        size = 2.0 ** min(i, 30 - i)
        slot = (1 if p < page else 3) * page + p % page
        check(None, bf(size * r.standard_normal((1, 2, 64))), bf(size * r.standard_normal((1, 2, 64))), [p], [slot],
              ref.frequencies(64), cache)


def test_tiny_zero_and_huge_values():
    r = np.random.default_rng(6)
    base = r.standard_normal((7, 1, 64))
    size = np.array([0.0, 1e-38, 1e-30, 1e-10, 1.0, 1e30, 3e38])[:, None, None]
    x = bf(np.clip(base, -1, 1) * size)
    check(None, x, x.clone(), list(range(7)), [16 * i for i in range(7)], [], make_cache(r, 7, 1, 16, 64))
    # growing over the whole range within one page
    cache = make_cache(r, 2, 1, 16, 64)
    for i in range(7):
        check(None, x[i:i + 1], x[i:i + 1].clone(), [i], [16 + i], [], cache)


def test_infinities_and_nan_are_coded_as_nan():
    r = np.random.default_rng(7)
    x = r.standard_normal((5, 2, 64))
    x[1, 0, 3], x[2, 1, 5], x[4, 0, :] = np.inf, -np.inf, np.nan
    check(None, bf(x), bf(x), list(range(5)), [4 + i for i in range(5)], [], make_cache(r, 2, 2, 16, 64))


def test_padding_and_slots_outside_the_cache_are_not_written():
    r = np.random.default_rng(8)
    slots = [-1, 3, -1, 20, 21, 2 ** 40, 4 * 16, 4 * 16 - 1, -2 ** 50]
    check(bf(r.standard_normal((9, 2, 128))), bf(r.standard_normal((9, 1, 128))), bf(r.standard_normal((9, 1, 128))),
          list(range(9)), slots, ref.frequencies(32), make_cache(r, 4, 1, 16, 128))


def test_whole_and_split_prompts_agree_where_scales_do():
    """A prompt written at once, and token by token: equal wherever the page's scale came out equal."""
    r = np.random.default_rng(9)
    k, v = bf(r.standard_normal((50, 2, 64))), bf(r.standard_normal((50, 2, 64)))
    a, b = make_cache(r, 5, 2, 16, 64), None
    b = [x.clone() for x in a]
    pos, slots = list(range(50)), list(range(16, 66))
    check(None, k, v, pos, slots, ref.frequencies(64), a)
    for i in range(50):
        check(None, k[i:i + 1], v[i:i + 1], pos[i:i + 1], slots[i:i + 1], ref.frequencies(64), b)
    assert torch.equal(a[2], b[2]) and torch.equal(a[3], b[3])
    x, y = (ref.values(c[0]) for c in (a, b))
    small = 2.0 ** -6                       # below it codes lose bits when a scale grows
    assert (np.abs(x - y) <= np.where(np.abs(x) < 2 * small, 2.0 ** -9, 0)).all()


def test_cache_past_4_gib():
    """Page numbers whose byte offsets pass 2^32, k and v."""
    hk, page, d = 8, 64, 256
    pages = 2 ** 32 // (hk * page * d) + 40
    k = torch.zeros(pages, hk, page, d, dtype=torch.uint8, device="cuda").view(F8)
    v = torch.zeros(pages, hk, d, page, dtype=torch.uint8, device="cuda").view(F8)
    ks, vs = (torch.zeros(pages, hk, device="cuda") for _ in range(2))
    r = np.random.default_rng(10)
    last = pages - 1
    slots = torch.tensor([last * page + 5, last * page + 6, 3], dtype=torch.int64, device="cuda")
    x = bf(r.standard_normal((3, hk, d)))
    ks[last], vs[last] = 2.0 ** -8, 2.0 ** -8
    gdn.gdn_rope_append_kv8(None, x, x.clone(), torch.zeros(3, dtype=torch.int32, device="cuda"), slots, None, None, k, v, ks, vs)
    torch.cuda.synchronize()
    for at, rows in ((last, [(5, 0), (6, 1)]), (0, [(3, 2)])):
        for off, t in rows:
            for h in range(hk):
                for c, sc in ((k[at, h, off], ks[at, h]), (v[at, h, :, off], vs[at, h])):
                    err = (c.float() * sc - x[t, h].float()).abs()
                    assert (err <= x[t, h].float().abs() * 2.0 ** -4 + sc * 2.0 ** -10).all()
    touched = (k.view(torch.uint8).view(pages, -1) != 0).any(1).nonzero().flatten().tolist()
    assert touched == [0, last]


def test_on_a_stream_of_its_own_and_in_a_graph():
    r = np.random.default_rng(11)
    pos, slots = runs(r, [(5, 1), (0, 37), (100, 1)], 16, 12)
    T = len(pos)
    q, k, v = bf(r.standard_normal((T, 4, 64))), bf(r.standard_normal((T, 2, 64))), bf(r.standard_normal((T, 2, 64)))
    cache = make_cache(r, 12, 2, 16, 64)
    start = [c.clone() for c in cache]
    args = (torch.tensor(pos, dtype=torch.int32, device="cuda"), torch.tensor(slots, device="cuda"),
            torch.tensor(ref.frequencies(64), device="cuda"))
    qo = torch.empty_like(q)
    gdn.gdn_rope_append_kv8(q, k, v, *args, qo, *cache)
    torch.cuda.synchronize()
    want = [qo.clone()] + [c.clone() for c in cache]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.default_stream())
        for c, c0 in zip(cache, start):
            c.view(torch.uint8).copy_(c0.view(torch.uint8))
        gdn.gdn_rope_append_kv8(q, k, v, *args, qo, *cache)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gdn.gdn_rope_append_kv8(q, k, v, *args, qo, *cache)
    for _ in range(3):
        for x, w in zip([qo] + cache, want):
            assert torch.equal(x.view(torch.uint8), w.view(torch.uint8))
        for c, c0 in zip(cache, start):
            c.view(torch.uint8).copy_(c0.view(torch.uint8))
        qo.zero_()
        g.replay()
        torch.cuda.synchronize()
