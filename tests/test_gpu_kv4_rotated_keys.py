"""GPU checks that gdn_rope_append_kv4 rotates keys in 64 bits and rounds them once before their codes,
for all head sizes, partly rotated heads, both layouts, with q, and one and two tokens per workgroup.

Keys are chosen so that a pair's first rotated element lies within four fp32 steps of the middle of two codes: products in
fp32 would move many of them to the other side."""
import numpy as np
import pytest
import torch

import kv4_ref as kv4
import serving_ref as ref
from test_gpu_kv4_append import bf, make_cache, numpy_of

import gated_deltanet_token_amd as gdn

MIDDLES = np.array([0.25, 0.75, 1.25, 1.75, 2.5])
STEPS = np.arange(-24, 25)


def bf16(x):
    return np.where(x == 0, 0.0, kv4.bf16(np.where(x == 0, 1.0, x)))


def near_middles(r, c, s):
    """Pairs (a, b) of bf16 values for cosines c and sines s [T][H][n], of scale 1 together: every eighth pair has the
    largest elements, 3.6 to 6.8.  Also which first elements lie next to a middle."""
    shape = c.shape
    p, q = r.uniform(3.7, 4.8, shape), r.uniform(3.7, 4.8, shape) * r.choice([-1, 1], shape)
    m2 = c * c + s * s
    top = bf16((p * c + q * s) / m2), bf16((q * c - p * s) / m2)
    a, b = bf16(r.standard_normal(shape)), bf16(r.standard_normal(shape))
    near = np.zeros(shape, bool)
    least = np.full(shape, 4.0)
    for m in MIDDLES:
        usable = (np.abs(c) > m / 2.9) & (np.abs(s) > 0.05)
        a0 = bf16(np.where(usable, m / np.where(usable, c, 1), 1.0))
        ulp = np.exp2(np.floor(np.log2(np.abs(a0))) - 7)
        for k in STEPS:
            x = bf16(a0 + k * ulp)
            y = bf16(np.where(usable, (x * c - m) / np.where(usable, s, 1), 0.0))
            off = np.abs(x * c - y * s - m) / np.spacing(np.float32(m) * np.float32(0.999))      # in fp32 steps
            better = usable & (off > 0.55) & (off < least) & (np.abs(y) > 2.0 ** -20)
            a, b, least, near = np.where(better, x, a), np.where(better, y, b), np.where(better, off, least), near | better
    at = np.arange(shape[-1]) % 8 == 0
    return np.where(at, top[0], a), np.where(at, top[1], b), near & ~at


def heads(a, b, d, rot, interleaved, r):
    x = r.uniform(-3, 3, (*a.shape[:2], d))
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    x[..., i], x[..., j] = a, b
    x[..., rot:] = bf16(x[..., rot:])
    x[..., rot::32] = 5.0
    return x, i, j


CASES = [(64, 64, False, 70), (64, 16, True, 70), (128, 48, False, 1), (128, 128, True, 300), (128, 64, False, 1500),
         (256, 64, False, 33), (256, 256, True, 1030), (256, 256, False, 200), (256, 80, False, 1024)]


def case(d, rot, interleaved, T):
    r = np.random.default_rng(d + rot + T)
    hk, m = 2, 1.1
    pos, freq = r.integers(1000, 100000, T), ref.frequencies(rot)
    ang = pos[:, None].astype(np.float64) * np.asarray(freq)
    c, s = (np.broadcast_to((m * f(ang))[:, None], (T, hk, rot // 2)) for f in (np.cos, np.sin))
    a, b, near = near_middles(r, c, s)
    k, i, j = heads(a, b, d, rot, interleaved, r)
    want = ref.rotate(k, pos, freq, m, interleaved)
    return r, hk, m, pos, freq, c, s, a, b, near, k, i, j, want


@pytest.mark.parametrize("d,rot,interleaved,T", CASES)
def test_products_in_fp32_would_be_seen(d, rot, interleaved, T):
    """The inputs' own check, on the CPU: rounded once, a first element is on its side of the middle; with sines, cosines and
    products in fp32 1 to 9 of 100 are not."""
    r, hk, m, pos, freq, c, s, a, b, near, k, i, j, want = case(d, rot, interleaved, T)
    assert near.sum() >= max(2, T * hk * rot // 32) and (np.abs(want) < 6.9).all()
    once = kv4.e2m1(want[..., i].astype(np.float32))
    f = lambda x: np.asarray(x).astype(np.float32).astype(np.float64)                          # noqa: E731
    plain = kv4.e2m1(f(a * f(c) - f(b * f(s))))
    assert (once != plain)[near].sum() >= max(1, near.sum() // 100)


@pytest.mark.gpu
@pytest.mark.parametrize("d,rot,interleaved,T", CASES)
def test_keys_next_to_the_middle_of_two_codes(d, rot, interleaved, T):
    """Angles up to 2^17 are off by 3 2^-53 of themselves and numpy's by one more, sines and cosines by less than
    that: 2^-34 (|a| + |b|) times the rope scale before the rounding to fp32."""
    r, hk, m, pos, freq, c, s, a, b, near, k, i, j, want = case(d, rot, interleaved, T)
    page, pages, hq = 16, -(-T // 16) + 1, 3
    cache = make_cache(r, pages, hk, page, d)
    q, v, kt = bf(r.standard_normal((T, hq, d))), bf(r.standard_normal((T, hk, d))), bf(k)
    assert np.array_equal(ref.values(kt), k)
    q_out = torch.full_like(q, 99.0)
    t = lambda x, dtype: torch.tensor(x, dtype=dtype, device="cuda")                           # noqa: E731
    gdn.gdn_rope_append_kv4(q, kt, v, t(pos, torch.int32), t(np.arange(T), torch.int64), t(np.asarray(freq), torch.float64), q_out, *cache,
                            interleaved=interleaved, rope_scale=m)
    torch.cuda.synchronize()
    kc, _, ks, _ = numpy_of(cache)
    codes = kc.swapaxes(1, 2).reshape(pages * page, hk, d)[:T]
    assert (ks.swapaxes(1, 2).reshape(pages * page, hk, d // 32)[:T] == 127).all()
    x, y = want[..., i], want[..., j]
    off = np.zeros(want.shape)
    off[..., i] = off[..., j] = 2.0 ** -33 * np.hypot(x, y)          # |a| + |b| <= sqrt 2 of it, rotation keeps it
    low, high = (kv4.VALUES[kv4.e2m1((want + sign * off).astype(np.float32))] for sign in (-1, 1))
    got = kv4.VALUES[codes]
    assert ((got >= low) & (got <= high)).all(), "%d codes" % ((got < low) | (got > high)).sum()
    assert (low != high).mean() < 1e-3
    qr = ref.values(q)
    qw = ref.rotate(qr, pos, freq, m, interleaved)
    big = np.abs(qr).max(-1, keepdims=True) * 2 * m
    assert (np.abs(ref.values(q_out) - qw) <= np.abs(qw) * 2.0 ** -8 + big * 2.0 ** -22).all()
