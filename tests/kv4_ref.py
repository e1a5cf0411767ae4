"""The 4-bit paged cache in plain 64-bit numpy on the CPU, from its definition:
what the GPU tests compare with."""
import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
VALUES = np.concatenate([MAGNITUDES, -MAGNITUDES])
LEAST = 2.0 ** -100


def e2m1(x):
    """Codes of the nearest values, ties to the even code; magnitudes above 6 become 6."""
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    lo = np.clip(np.searchsorted(MAGNITUDES, a, side="right") - 1, 0, 6)
    middle = (MAGNITUDES[lo] + MAGNITUDES[lo + 1]) / 2
    n = np.where((a > middle) | ((a == middle) & (lo % 2 == 1)), lo + 1, lo)
    return (n + 8 * np.signbit(x)).astype(np.uint8)


def key_exponent(m):
    """Of the scale of 32 elements whose largest magnitude is m (finite)."""
    m = np.asarray(m, np.float64)
    f, e = np.frexp(m)                                   # m = f 2^e, f from 0.5 to 1
    return np.where(m > 0, np.maximum(e - 3 + (f >= 0.875), -100), -100)


def bf16(x):
    """x rounded to the nearest bf16 value (normal range), ties to even."""
    f, e = np.frexp(np.asarray(x, np.float64))
    return np.ldexp(np.round(f * 256) / 256, e)


def value_scale(m):
    return np.maximum(bf16(np.asarray(m, np.float64) / 6), LEAST)


def quantise_k(x):
    """x [..., D] -> codes [..., D], scale bytes [..., D / 32]."""
    b = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, 32)
    fine = np.isfinite(b).all(-1)
    e = key_exponent(np.abs(np.where(fine[..., None], b, 0.0)).max(-1))
    codes = e2m1(np.where(fine[..., None], b, 0.0) / np.exp2(e)[..., None])
    return codes.reshape(x.shape), np.where(fine, e + 127, 255).astype(np.uint8)


def quantise_v(x):
    """x [..., D] -> codes [..., D], scales [...] (values)."""
    x = np.asarray(x, np.float64)
    fine = np.isfinite(x).all(-1)
    s = value_scale(np.abs(np.where(fine[..., None], x, 0.0)).max(-1))
    return e2m1(np.where(fine[..., None], x, 0.0) / s[..., None]), np.where(fine, s, np.nan)


def key_values(codes, scale):
    """Codes [..., D] and scale bytes [..., D / 32] -> values."""
    s = np.where(scale == 255, np.nan, np.exp2(scale.astype(np.float64) - 127))
    return VALUES[codes] * np.repeat(s, 32, axis=-1)


def value_values(codes, scale):
    with np.errstate(invalid="ignore"):
        return VALUES[codes] * np.asarray(scale, np.float64)[..., None]


# the arrays as they lie in memory; codes [pages][hk][page][D]

def pack_k(codes):
    return (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)


def unpack_k(packed):
    return np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)


def pack_v(codes):
    n, hk, page, d = codes.shape
    t = codes.reshape(n, hk, page // 16, 16, d).transpose(0, 1, 2, 4, 3)
    return np.ascontiguousarray(pack_k(t))


def unpack_v(packed):
    n, hk, g, d, _ = packed.shape
    return unpack_k(packed).transpose(0, 1, 2, 4, 3).reshape(n, hk, g * 16, d)


def pack_k_scale(scale):
    """[pages][hk][page][D / 32] -> [pages][hk][D / 32][page]"""
    return np.ascontiguousarray(scale.transpose(0, 1, 3, 2))


# q in three e2m3 parts

def e2m3(x):
    """The nearest values of 2 exponent and 3 mantissa bits (ties to even, at most 7.5)."""
    x = np.asarray(x, np.float64)
    step = np.exp2(np.floor(np.log2(np.clip(np.abs(x), 1.0, None))) - 3)
    return np.clip(np.round(x / step) * step, -7.5, 7.5)


def split(x):
    """The three parts' sum of 32 elements each, x [..., 32]."""
    s = np.exp2(np.floor(np.log2(np.maximum(np.abs(x).max(-1, keepdims=True), 2.0 ** -110))) - 1)
    got = np.zeros_like(x)
    for unit in (s, s / 32, s / 1024):
        got = got + e2m3((x - got) / unit) * unit
    return got
