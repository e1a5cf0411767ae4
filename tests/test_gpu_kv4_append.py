"""GPU checks of gdn_rope_append_kv4 against its definition in 64 bits.

Values, unrotated elements and every scale of theirs: equality.  Rotated elements of q:
sines and cosines rounded to fp32 (2^-24 of each), a product and a sum of two
rounded (2^-24 each) are off by at most 2^-24 (2 |a c| + 3 |b s|) < 3 2^-24 (|a c| +
|b s|), and a subnormal step; q has to be within that and half a bf16 step (2^-8).
Keys are held to the same here: a code has to be that of some number this close to the
exact one, a scale that of a magnitude this close to the largest.  That they are rotated in
64 bits and rounded once is checked by test_rotated_keys_are_rounded_once_before_their_codes
and, for all shapes, in test_gpu_kv4_rotated_keys.py."""
import numpy as np
import pytest
import torch

import gated_deltanet_token_amd as gdn
import kv4_ref as kv4
import serving_ref as ref

pytestmark = pytest.mark.gpu


def bf(a):
    return torch.tensor(np.asarray(a, np.float32), device="cuda").to(torch.bfloat16)


def make_cache(r, pages, hk, page, d):
    """A cache of any content."""
    u8 = lambda *s: torch.tensor(r.integers(0, 256, s, dtype=np.uint8), device="cuda")         # noqa: E731
    return [u8(pages, hk, page, d // 2), u8(pages, hk, page // 16, d, 8), u8(pages, hk, d // 32, page),
            u8(pages, hk, page, 2).view(torch.bfloat16).squeeze(-1)]


def numpy_of(cache):
    """codes of k and v [pages][hk][page][D], k's scale bytes [pages][hk][page][D / 32], v's scales as their bits"""
    k, v, ks, vs = cache
    return (kv4.unpack_k(k.cpu().numpy()), kv4.unpack_v(v.cpu().numpy()), ks.cpu().numpy().transpose(0, 1, 3, 2),
            vs.contiguous().view(torch.int16).cpu().numpy().view(np.uint16))


def bits(x):
    """of bf16 values"""
    return torch.tensor(np.asarray(x)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def rotation_error(x, pos, freq, rope_scale, interleaved):
    """3 2^-24 (|a c| + |b s|) of each element."""
    n = len(freq)
    err = np.zeros(x.shape)
    if n:
        ang = np.asarray(pos, np.float64)[:, None] * np.asarray(freq)[None]
        c, s = (np.abs(rope_scale * f(ang))[:, None] for f in (np.cos, np.sin))
        i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
        a, b = np.abs(x[..., i]), np.abs(x[..., j])
        err[..., i], err[..., j] = a * c + b * s, b * c + a * s
        err = err * 3 * 2.0 ** -24 + np.where(err > 0, 2.0 ** -148, 0.0)
    return err


def check_key(codes, scale, x, err):
    """One [T][D / 32] block array's codes [.., 32] and scale bytes against x and its error."""
    fine = np.isfinite(x).all(-1)
    assert (scale[~fine] == 255).all()
    x, err, codes, scale = x[fine], err[fine], codes[fine], scale[fine].astype(np.int64)
    m, em = np.abs(x).max(-1), err.max(-1)
    lo, hi = kv4.key_exponent(np.maximum(m - em, 0)), kv4.key_exponent(m + em)
    assert ((scale - 127 >= lo) & (scale - 127 <= hi)).all()
    s = np.exp2(scale - 127.0)[..., None]
    got = kv4.VALUES[codes]
    low, high = kv4.VALUES[kv4.e2m1((x - err) / s)], kv4.VALUES[kv4.e2m1((x + err) / s)]
    assert ((got >= low) & (got <= high)).all(), "%d codes" % ((got < low) | (got > high)).sum()
    exact = err == 0
    assert (codes[exact] == kv4.e2m1(x / s)[exact]).all()


def call(q, k, v, pos, slots, freq, cache, interleaved=False, rope_scale=1.0, q_out=None):
    f = torch.tensor(freq, dtype=torch.float64, device="cuda") if len(freq) else None
    gdn.gdn_rope_append_kv4(q, k, v, torch.tensor(pos, dtype=torch.int32, device="cuda"),
                            torch.tensor(slots, dtype=torch.int64, device="cuda"), f, q_out, *cache, interleaved=interleaved,
                            rope_scale=rope_scale)
    torch.cuda.synchronize()


def check(q, k, v, pos, slots, freq, cache, interleaved=False, rope_scale=1.0, q_out=None):
    before = numpy_of(cache)
    qr, kr, vr = (None if x is None else ref.values(x) for x in (q, k, v))
    if q is not None and q_out is None:
        q_out = torch.full(q.shape, 99.0, dtype=torch.bfloat16, device="cuda")
    call(q, k, v, pos, slots, freq, cache, interleaved, rope_scale, q_out)
    kc, vc, ks, vs = numpy_of(cache)
    pages, hk, page, d = kc.shape
    slots = np.asarray(slots)
    on = np.flatnonzero((slots >= 0) & (slots < pages * page))
    at, off = slots[on] // page, slots[on] % page
    with np.errstate(invalid="ignore"):
        krot, err = ref.rotate(kr, pos, freq, rope_scale, interleaved), rotation_error(kr, pos, freq, rope_scale, interleaved)
    # an fp32 overflow or a NaN operand is not finite there either
    blocks = lambda x: x[on].reshape(len(on), hk, d // 32, 32)                                  # noqa: E731
    check_key(kc[at, :, off].reshape(len(on), hk, d // 32, 32), ks[at, :, off], blocks(krot), np.nan_to_num(blocks(err)))
    codes, scale = kv4.quantise_v(vr[on])
    fine = np.isfinite(scale)
    assert np.array_equal(vs[at, :, off][fine], bits(scale)[fine]) and (vs[at, :, off][~fine] & 0x7fff > 0x7f80).all()
    assert np.array_equal(vc[at, :, off][fine], codes[fine])
    # nothing else has changed
    for got, was in zip((kc, vc, ks, vs), before):
        got[at, :, off] = was[at, :, off]
        assert np.array_equal(got, was)
    if q is not None:
        want, err = ref.rotate(qr, pos, freq, rope_scale, interleaved), rotation_error(qr, pos, freq, rope_scale, interleaved)
        assert (np.abs(ref.values(q_out) - want) <= (np.abs(want) + err) * 2.0 ** -8 + err + 2.0 ** -134).all()
    return q_out


def runs(r, spec, page, pages):
    """positions and slots of requests given as (context, new): pages at random ids."""
    ids = list(r.permutation(pages))
    pos, slots = [], []
    for c, n in spec:
        mine = [ids.pop() for _ in range(-(-(c + n) // page) - c // page)]
        for i in range(c, c + n):
            pos.append(i)
            slots.append(int(mine[i // page - c // page]) * page + i % page)
    return pos, slots


MIXED = [(5, 1), (16, 1), (31, 1), (1000, 1), (0, 70), (9, 40), (15, 17), (100, 3), (47, 1), (0, 1), (64, 128)]


@pytest.mark.parametrize("d,page,rot,interleaved", [
    (64, 16, 64, False), (64, 64, 16, True), (128, 32, 128, True), (128, 16, 48, False), (256, 16, 64, False), (256, 64, 256, False),
    (256, 32, 80, True), (128, 64, 0, False)])
@pytest.mark.parametrize("hq,hk", [(4, 2), (5, 5), (8, 1), (3, 3)])
def test_mixed_runs(d, page, rot, interleaved, hq, hk):
    r = np.random.default_rng(d + page + rot + hq)
    pos, slots = runs(r, MIXED, page, 40)
    T = len(pos)
    x = lambda h: bf(r.standard_normal((T, h, d)) * np.exp(r.standard_normal((T, h, 1))))       # noqa: E731
    check(x(hq), x(hk), x(hk), pos, slots, ref.frequencies(rot) if rot else [], make_cache(r, 40, hk, page, d), interleaved, 1.25)


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 600, 5000])
def test_numbers_of_tokens(n):
    """Decode rows and a prompt that fill windows of 64 tokens exactly, or one more or less."""
    r = np.random.default_rng(n)
    pos, slots = runs(r, [(int(c), 1) for c in r.integers(0, 200, n // 2)] + [(7, n - n // 2)], 16, n + 30)
    x = lambda h: bf(r.standard_normal((n, h, 64)))                                            # noqa: E731
    check(x(3), x(3), x(3), pos, slots, ref.frequencies(32), make_cache(r, n + 30, 3, 16, 64))


def test_columns_of_a_projection_q_in_place():
    r = np.random.default_rng(1)
    pos, slots = runs(r, MIXED, 16, 40)
    T, hq, hk, d = len(pos), 8, 2, 128
    qkv = bf(r.standard_normal((T, hq + 2 * hk + 1, d)))
    was = qkv.clone()
    q = qkv[:, :hq]
    freq = ref.frequencies(64)
    qr = ref.values(q)
    cache = make_cache(r, 40, hk, 16, d)
    call(q, qkv[:, hq:hq + hk], qkv[:, hq + hk:hq + 2 * hk], pos, slots, freq, cache, q_out=q)
    want, err = ref.rotate(qr, pos, freq, 1.0, False), rotation_error(qr, pos, freq, 1.0, False)
    assert (np.abs(ref.values(q) - want) <= (np.abs(want) + err) * 2.0 ** -8 + err).all()
    assert torch.equal(qkv[:, hq:], was[:, hq:]) and torch.equal(q[..., 64:], was[:, :hq, 64:])
    check(None, was[:, hq:hq + hk], was[:, hq + hk:hq + 2 * hk], pos, slots, freq, make_cache(r, 40, hk, 16, d))


def test_far_positions_scaled():
    """Positions of a million and more: angles in 64 bits."""
    r = np.random.default_rng(2)
    freq, m = gdn.gdn_rope_frequencies(128, 1e6, "yarn", 4.0, original_context=32768)
    pos = [2 ** 31 - 1, 10 ** 6, 131071, 65536, 2 ** 24 + 1]
    slots = [3, 100, 64, 33, 17]
    x = lambda h: bf(r.standard_normal((5, h, 128)))                                           # noqa: E731
    check(x(4), x(2), x(2), pos, slots, freq, make_cache(r, 8, 2, 16, 128), rope_scale=m)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotated_keys_are_rounded_once_before_their_codes(interleaved):
    """8 million elements, some of which lie closer to the middle of two codes than fp32 products
    are exact.  Angles up to 2^17 are off by 3 2^-53 of themselves and numpy's by one more, sines and
    cosines by less than that: 2^-34 (|a| + |b|) before the rounding to fp32."""
    r = np.random.default_rng(12)
    T, hk, d, page = 8192, 8, 128, 64
    freq, m = gdn.gdn_rope_frequencies(128, 1e6, "yarn", 4.0, original_context=32768)
    pos = r.integers(0, 2 ** 17, T)
    cache = make_cache(r, T // page, hk, page, d)
    x = bf(r.standard_normal((T, hk, d)))
    call(None, x, x.clone(), pos, np.arange(T), freq, cache, interleaved, m)
    kc, _, ks, _ = numpy_of(cache)
    codes, scale = (y.swapaxes(1, 2).reshape(T, hk, d // 32, 32) for y in (kc, ks[..., None].repeat(32, -1)))
    k = ref.values(x)
    want = ref.rotate(k, pos, freq, m, interleaved)
    a, b = (want[..., 0::2], want[..., 1::2]) if interleaved else (want[..., :64], want[..., 64:])
    off = 2.0 ** -33 * np.hypot(a, b)                                      # |a| + |b| <= sqrt 2 of it, rotation keeps it
    off = np.stack([off, off], -1).reshape(want.shape) if interleaved else np.concatenate([off, off], -1)
    s = np.exp2(scale - 127.0)
    low, high = (kv4.VALUES[kv4.e2m1((want + sign * off).astype(np.float32).astype(np.float64).reshape(s.shape) / s)] for sign in (-1, 1))
    got = kv4.VALUES[codes]
    assert ((got >= low) & (got <= high)).all(), "%d codes" % ((got < low) | (got > high)).sum()
    assert (low != high).mean() < 1e-6


@pytest.mark.parametrize("d", [64, 128, 256])
def test_every_significand_against_every_scale(d):
    """Values: largest magnitudes of all 128 significands, elements of all significands
    over their binades, ties of two codes among them.  Keys, unrotated: the same."""
    r = np.random.default_rng(3)
    sig = 1 + np.arange(128) / 128
    x = sig[None] * np.exp2(-np.arange(5))[:, None]                              # 640 magnitudes from 1/16 to 2
    T = 128 * (-(-640 // (d - 1)))
    rows = np.zeros((T, d))
    for t in range(T):
        top = sig[t % 128] * 2
        part = x.ravel()[(t // 128) * (d - 1):][:d - 1]
        rows[t, :len(part)] = np.minimum(part, top) * r.choice([-1, 1], len(part))
        rows[t, d - 1] = top
    rows = np.ldexp(rows, r.integers(-60, 60, (T, 1)))
    pages = -(-T // 16)
    v = bf(rows)[:, None]
    assert (ref.values(v)[:, 0] == rows).all()
    k = bf(np.stack([np.roll(rows, s, 1) for s in (0, 5)], 1))
    check(None, k, torch.cat([v, -v], 1), list(range(T)), list(range(T)), [], make_cache(r, pages, 2, 16, d))


def test_tiny_zero_and_huge_values():
    r = np.random.default_rng(4)
    T, d = 12, 64
    x = r.standard_normal((T, 2, d))
    for t, e in enumerate((-133, -126, -110, -100, -98, -97, 0, 60, 100, 120, 125, None)):
        x[t] = 0.0 if e is None else np.ldexp(x[t] / np.abs(x[t]).max(), e)
    x[6, 0, :32] = 0                                       # one block of zeros beside another
    check(None, bf(x), bf(x), list(range(T)), list(range(20, 20 + T)), [], make_cache(r, 4, 2, 16, d))


def test_infinities_and_nan_mark_their_block_or_head():
    r = np.random.default_rng(5)
    T, d = 20, 128
    k, v = bf(r.standard_normal((T, 2, d))), bf(r.standard_normal((T, 2, d)))
    k[3, 0, 5], k[7, 1, 127], k[8, 0, 64] = float("nan"), float("inf"), float("-inf")
    v[2, 0, 0], v[9, 1, 100], v[19, 1, 127] = float("nan"), float("inf"), float("-inf")
    check(None, k, v, list(range(T)), list(range(5, 5 + T)), [], make_cache(r, 2, 2, 16, d))


def test_padding_and_slots_outside_the_cache_are_not_written():
    r = np.random.default_rng(6)
    T, pages, page = 40, 3, 32
    slots = [-1, 5, 6, 7, -1, pages * page, 40, 41, 2 ** 40, -2 ** 40, 95, pages * page, 64, -1] + [-1] * (T - 14)
    x = lambda h: bf(r.standard_normal((T, h, 64)))                                            # noqa: E731
    check(x(2), x(2), x(2), list(range(T)), slots, ref.frequencies(64), make_cache(r, pages, 2, page, 64))


def test_a_prompt_token_by_token_is_the_same():
    """What a call stores does not depend on what else it stores, or on what was there."""
    r = np.random.default_rng(7)
    T, d, page = 75, 128, 32
    k, v = bf(r.standard_normal((T, 2, d))), bf(r.standard_normal((T, 2, d)))
    freq, slots = ref.frequencies(128), list(range(9, 9 + T))
    a, b = make_cache(r, 3, 2, page, d), make_cache(r, 3, 2, page, d)
    call(None, k, v, list(range(T)), slots, freq, a)
    for t in range(T):
        call(None, k[t:t + 1], v[t:t + 1], [t], slots[t:t + 1], freq, b)
    for x, y in zip(numpy_of(a), numpy_of(b)):
        x, y = (z.swapaxes(1, 2).reshape(3 * page, -1)[9:9 + T] for z in (x, y))
        assert np.array_equal(x, y)


def test_cache_past_4_gib():
    r = np.random.default_rng(8)
    hk, page, d = 4, 64, 256
    pages = 2 ** 33 // (hk * page * d) + 20
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")                          # noqa: E731
    cache = [u8(pages, hk, page, d // 2), u8(pages, hk, page // 16, d, 8), u8(pages, hk, d // 32, page),
             torch.zeros(pages, hk, page, dtype=torch.bfloat16, device="cuda")]
    T = 50
    k, v = bf(r.standard_normal((T, hk, d))), bf(r.standard_normal((T, hk, d)))
    first = (pages - 2) * page + 40
    call(None, k, v, list(range(T)), list(range(first, first + T)), [], cache)
    tail = [c[-2:].clone() for c in cache]
    small = [torch.zeros_like(c) for c in tail]
    call(None, k, v, list(range(T)), list(range(40, 40 + T)), [], small)
    for a, b, c in zip(tail, small, cache):
        assert torch.equal(a, b) and not c[:-2].view(torch.uint8).any()


def test_on_a_stream_of_its_own_and_in_a_graph():
    r = np.random.default_rng(9)
    pos, slots = runs(r, MIXED, 16, 40)
    T = len(pos)
    q, k, v = (bf(r.standard_normal((T, h, 128))) for h in (4, 2, 2))
    freq = torch.tensor(ref.frequencies(64), device="cuda")
    p, s = torch.tensor(pos, dtype=torch.int32, device="cuda"), torch.tensor(slots, device="cuda")
    start = make_cache(r, 40, 2, 16, 128)
    want, q_want = [c.clone() for c in start], torch.empty_like(q)
    gdn.gdn_rope_append_kv4(q, k, v, p, s, freq, q_want, *want)
    side, got, q_out = torch.cuda.Stream(), [c.clone() for c in start], torch.empty_like(q)
    torch.cuda.synchronize()
    gdn.gdn_rope_append_kv4(q, k, v, p, s, freq, q_out, *got, stream=side)
    side.synchronize()
    same = lambda: torch.equal(q_out, q_want) and all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))   # noqa: E731
                                                      for a, b in zip(got, want))
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_rope_append_kv4(q, k, v, p, s, freq, q_out, *got)
    for _ in range(3):
        for a, b in zip(got, start):
            a.copy_(b)
        q_out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same()
