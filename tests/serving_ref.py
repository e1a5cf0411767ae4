"""The attention layers' operators and the block norms in plain 64-bit
numpy / torch on the CPU, from their formulas: what the GPU tests compare
with."""
import math

import numpy as np
import torch

F8 = torch.float8_e4m3fn


def tables(ctx, new, free, num_free, table, page, T, n_chunks):
    """query_start_loc, seq_lens, positions, slots, table, chunks, counts; one
    request and one token at a time."""
    table = table.copy()
    max_pages = table.shape[1]
    num_free = min(max(num_free, 0), len(free))
    qsl, seq, pos, slots, chunks = [0], [], [], [], []
    got = missing = 0
    for s, (c, n) in enumerate(zip(ctx, new)):
        c, n = max(int(c), 0), max(int(n), 0)
        have, want = -(-c // page), -(-(c + n) // page)
        for i in range(have, want):
            if i < max_pages and got < num_free:
                table[s, i] = free[num_free - 1 - got]
                got += 1
            else:
                missing += 1
                if i < max_pages:
                    table[s, i] = -1
        for i in range(n):
            p, at = c + i, (c + i) // page
            pos.append(p)
            slots.append(int(table[s, at]) * page + p % page if at < max_pages and table[s, at] >= 0 else -1)
        chunks += [(s, i) for i in range(-(-n // 8))]
        qsl.append(qsl[-1] + n)
        seq.append(c + n)
    counts = [len(pos), len(chunks), got, missing]
    pos, slots, chunks = (x + pad * max(0, m - len(x)) for x, pad, m in
                          ((pos, [-1], T), (slots, [-1], T), (chunks, [(-1, 0)], n_chunks)))
    return (np.array(qsl, np.int32), np.array(seq, np.int32), np.array(pos[:T], np.int32), np.array(slots[:T], np.int64), table,
            np.array(chunks[:n_chunks], np.int32).reshape(-1, 2), np.array(counts, np.int32))


def e4m3(x):
    """Nearest e4m3 value (ties to even) of |x| <= 448; anything not finite: NaN."""
    x = np.asarray(x, np.float64)
    fine = np.isfinite(x)
    y = np.where(fine, x, 0.0)
    _, e = np.frexp(y)
    step = np.exp2(np.maximum(e - 1, -6) - 3)
    return np.where(fine, np.round(y / step) * step, np.nan)


def block_scale(amax):
    s = 2.0 ** -100
    while amax > 448 * s:
        s *= 2
    return s


def rotate(x, pos, freq, rope_scale, interleaved):
    """x [T][H][D] in 64 bits, rotated."""
    x = np.array(x, np.float64)
    n = len(freq)
    if not n:
        return x
    ang = np.asarray(pos, np.float64)[:, None] * np.asarray(freq)[None]
    c, s = rope_scale * np.cos(ang)[:, None], rope_scale * np.sin(ang)[:, None]
    i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    a, b = x[..., i].copy(), x[..., j].copy()
    x[..., i], x[..., j] = a * c - b * s, b * c + a * s
    return x


def append(x, slots, codes, scale):
    """codes [pages][H][page][D] (values) and scale [pages][H] with x [T][H][D]
    written at slots; new arrays."""
    codes, scale = codes.astype(np.float64).copy(), scale.astype(np.float64).copy()
    pages, H, page, _ = codes.shape
    t, T = 0, len(slots)
    while t < T:
        if slots[t] < 0 or slots[t] >= pages * page:
            t += 1
            continue
        p, off = divmod(int(slots[t]), page)
        n = 1
        while t + n < T and off + n < page and slots[t + n] == slots[t] + n:
            n += 1
        for h in range(H):
            y = x[t:t + n, h]
            fine = np.abs(y[np.isfinite(y)])
            now = block_scale(fine.max() if fine.size else 0.0)
            if off:
                now = max(now, scale[p, h])
                if now != scale[p, h]:
                    codes[p, h, :off] = e4m3(codes[p, h, :off] * (scale[p, h] / now))
            codes[p, h, off:off + n] = e4m3(y / now)
            scale[p, h] = now
        t += n
    return codes, scale


def attention(q, k, v, ks, vs, table, seq, qsl, scale, causal=True, window=0):
    """o [T][HQ][D] and sum_j w_j |v_j| (what a relative error of the weights
    scales with); k values [pages][HK][page][D], v [pages][HK][D][page]; rows
    that no request owns: NaN and -1."""
    q = q.astype(np.float64)
    T, HQ, D = q.shape
    pages, HK, page, _ = k.shape
    G = HQ // HK
    o, mag = np.full((T, HQ, D), np.nan), np.full((T, HQ, D), -1.0)
    for s in range(len(seq)):
        a, b = min(max(qsl[s], 0), T), min(max(qsl[s + 1], 0), T)
        full = max(int(seq[s]), 0)
        L = min(full, table.shape[1] * page)
        j = np.arange(L)
        ids = table[s][j // page] if L else np.zeros(0, np.int64)
        known = (ids >= 0) & (ids < pages)
        ids = np.where(known, ids, 0)
        for t in range(a, b):
            p = full - (b - a) + (t - a)
            see = known.copy()
            if causal:
                see &= j <= p
            if window:
                see &= j > p - window
            o[t], mag[t] = 0.0, 0.0
            if not see.any():
                continue
            js, pg = j[see], ids[see]
            for h in range(HK):
                K = k[pg, h, js % page] * ks[pg, h][:, None].astype(np.float64)
                V = v[pg, h][np.arange(len(js)), :, js % page] * vs[pg, h][:, None].astype(np.float64)
                for g in range(h * G, h * G + G):
                    x = scale * (K @ q[t, g])
                    w = np.exp(x - x.max())
                    w /= w.sum()
                    o[t, g], mag[t, g] = w @ V, w @ np.abs(V)
    return o, mag


def rms(x, eps):
    return 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def sigmoid(z):
    return 1.0 / (1.0 + np.exp(-z))


def values(t):
    """A tensor's values as float64 numpy."""
    return t.detach().cpu().to(torch.float64).numpy()


def quantised(x):
    """Codes (values) and scales of x [pages][H][...] with one scale per page and head."""
    x = np.asarray(x, np.float64)
    sc = np.array([[block_scale(np.abs(x[p, h]).max()) for h in range(x.shape[1])] for p in range(x.shape[0])])
    return e4m3(x / sc.reshape(sc.shape + (1,) * (x.ndim - 2))), sc


def frequencies(rot, base=10000.0):
    return np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])


def turns(f, original):
    return original * f / (2 * math.pi)
