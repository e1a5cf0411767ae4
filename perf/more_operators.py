"""What the operators of the 4-bit paged cache cost, and what they compute.

Three operators of an attention layer whose keys and values are held in 4 bits, each through its public entry points (``own``)
or in plain torch:

  update     gdn_rope_append_kv4 and gdn_paged_read_kv4: rotary positions on q and k, the step's k and v quantised into the
             cache, and what the cache now holds of them read back (a layer that attends to its new tokens as they are stored)
  read       gdn_paged_read_kv4: ranges of keys and values of a batch of requests out of the cache, as packed bf16 rows
  attention  gdn_paged_attention_kv4: attention of the step's tokens over the cache, decode rows and prompt chunks

The cache holds e2m1 codes (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign), two to a byte, the first in the low half:

  k_cache  [pages][kv heads][page][head dim / 2]      two elements of a key to a byte
  k_scale  [pages][kv heads][head dim / 32][page]     e8m0 (a power of two, biased by 127; 255: NaN) of 32 elements of a key
  v_cache  [pages][kv heads][page / 16][head dim][8]  an element's codes of 16 neighbouring tokens
  v_scale  [pages][kv heads][page]                    bf16, of a token's value

A key's 32 elements are scaled by the power of two that belongs to their largest magnitude rounded to one bit behind the leading
one (the largest code is then met by 3.5 to 7), a value by a sixth of its largest magnitude.
"""
import math
import random

import torch

own = False


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    # head shapes: 16 q / 4 kv heads of 256 with 64 rotated elements, and 32 / 8 of 128
    small = {"hq": 16, "hk": 4, "d": 256, "page": 16}
    wide = {"hq": 32, "hk": 8, "d": 128, "page": 32}
    full = {"causal": True, "window": 0}
    return [
        # a decode step at concurrency 32 (1,024-token prompts, up to 128 new tokens): its new keys and values
        {"name": "update_decode_32", "op": "update", "decodes": 32, "ctx_lo": 1024, "ctx_hi": 1151, "chunks": 0, "chunk_tokens": 0,
         "chunk_ctx": 0, "mix": 1, **small, "rot": 64, "interleaved": False, "yarn": False},
        # a mixed step at the 2,048-token budget: 29 decode rows and three prompt chunks
        {"name": "update_mixed_2048", "op": "update", "decodes": 29, "ctx_lo": 1024, "ctx_hi": 1151, "chunks": 3,
         "chunk_tokens": 2019, "chunk_ctx": 700, "mix": 3, **small, "rot": 64, "interleaved": False, "yarn": False},
        # long prompts read in at once, whole heads rotated in the interleaved layout, scaled for long contexts
        {"name": "update_prefill_16384", "op": "update", "decodes": 0, "ctx_lo": 0, "ctx_hi": 0, "chunks": 8,
         "chunk_tokens": 16384, "chunk_ctx": 100000, "mix": 4, **wide, "rot": 128, "interleaved": True, "yarn": True},
        # the tail of one request's prompt behind the pages that it shares with others: the smallest call, all latency
        {"name": "read_tail_37", "op": "read", "requests": 1, "rows": 37, "start_hi": 1000, "mix": 7, **small},
        # the cached contexts of a step's prompt chunks, ragged, from the middle of pages on
        {"name": "read_contexts_30000", "op": "read", "requests": 29, "rows": 30000, "start_hi": 500, "mix": 8, **small},
        # one long context, moved to another engine or another kind of cache
        {"name": "read_context_131071", "op": "read", "requests": 1, "rows": 131071, "start_hi": 0, "mix": 9, **wide},
        # the decode step's attention
        {"name": "attention_decode_32", "op": "attention", "decodes": 32, "ctx_lo": 1024, "ctx_hi": 1151, "chunks": 0,
         "chunk_tokens": 0, "chunk_ctx": 0, "mix": 1, **small, **full},
        # a busy server's decode step: 200 requests of all lengths
        {"name": "attention_decode_200", "op": "attention", "decodes": 200, "ctx_lo": 1, "ctx_hi": 8000, "chunks": 0,
         "chunk_tokens": 0, "chunk_ctx": 0, "mix": 2, **wide, **full},
        # a few requests with very long contexts of unlike lengths
        {"name": "attention_decode_long", "op": "attention", "decodes": 5, "ctx_lo": 40000, "ctx_hi": 131071, "chunks": 0,
         "chunk_tokens": 0, "chunk_ctx": 0, "mix": 5, **wide, **full},
        # the mixed step's attention
        {"name": "attention_mixed_2048", "op": "attention", "decodes": 29, "ctx_lo": 1024, "ctx_hi": 1151, "chunks": 3,
         "chunk_tokens": 2019, "chunk_ctx": 700, "mix": 3, **small, **full},
        # one long prompt
        {"name": "attention_prefill_8192", "op": "attention", "decodes": 0, "ctx_lo": 0, "ctx_hi": 0, "chunks": 1,
         "chunk_tokens": 8192, "chunk_ctx": 0, "mix": 6, **wide, **full},
        # heads of 64 with a window, prompts that continue cached contexts, large pages
        {"name": "attention_window_5000", "op": "attention", "decodes": 11, "ctx_lo": 500, "ctx_hi": 9000, "chunks": 4,
         "chunk_tokens": 5000, "chunk_ctx": 6000, "mix": 10, "hq": 24, "hk": 8, "d": 64, "page": 64, "causal": True, "window": 1024},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("update", "read", "attention", "attention"))
    hk = rng.choice((1, 2, 4, 8))
    c = {"op": op, "hq": hk * rng.choice((1, 2, 4, 5, 8) if hk < 8 else (1, 2, 3, 4)), "hk": hk, "d": rng.choice((64, 128, 256)),
         "page": rng.choice((16, 32, 64)), "mix": rng.randrange(1 << 20)}
    if op == "read":
        rows = _log(rng, 1, 131072 * 8 * 128 // (hk * c["d"]) if hk * c["d"] > 1024 else 131072)
        return {**c, "requests": min(rows, _log(rng, 1, 200)), "rows": rows, "start_hi": rng.choice((0, 0, 40, 3000))}
    form = rng.choice(("decode", "decode", "mixed", "prefill"))
    c.update(decodes=0, ctx_lo=1, ctx_hi=1, chunks=0, chunk_tokens=0, chunk_ctx=0)
    if op == "update":
        if form != "prefill":
            c.update(decodes=_log(rng, 1, 400), ctx_hi=_log(rng, 16, 4096))
        if form != "decode":
            c.update(chunks=rng.randrange(1, 9), chunk_tokens=_log(rng, 16, 8192), chunk_ctx=rng.choice((0, 3000)))
        c.update(rot=rng.choice((c["d"], c["d"] // 2, c["d"] // 4)), interleaved=rng.random() < 0.5, yarn=rng.random() < 0.5)
        return c
    if form == "decode":
        c["decodes"] = _log(rng, 1, 200)
        c["ctx_hi"] = _log(rng, 16, min(131072, 400000 // c["decodes"]))
        c["ctx_lo"] = rng.choice((1, max(1, c["ctx_hi"] // 2)))
    elif form == "mixed":
        c.update(decodes=_log(rng, 1, 30), ctx_hi=_log(rng, 16, 2048), chunks=rng.randrange(1, 4), chunk_tokens=_log(rng, 16, 1500),
                 chunk_ctx=rng.choice((0, 900)))
    else:
        c.update(chunks=rng.randrange(1, 4), chunk_tokens=_log(rng, 16, 4000), chunk_ctx=rng.choice((0, 1000)))
    c["causal"] = rng.random() < 0.85
    c["window"] = rng.choice((0, 0, 0, _log(rng, 16, 1024)))
    return c


def _lengths(case):
    """(context, new) tokens of each request, decode rows first; of a read: (first key, rows)."""
    r = random.Random(case["mix"])
    if case["op"] == "read":
        n, left = case["requests"], case["rows"]
        got = []
    else:
        n, left = case["chunks"], case["chunk_tokens"]
        got = [(r.randint(case["ctx_lo"], max(case["ctx_lo"], case["ctx_hi"])), 1) for _ in range(case["decodes"])]
    for i in range(n):
        rest = n - 1 - i
        take = left if not rest else max(1, min(left - rest, int(r.uniform(0.5, 1.5) * left / (rest + 1))))
        if case["op"] == "read":
            got.append((r.randint(0, case["start_hi"]), take))
        else:
            got.append((r.randint(0, case["chunk_ctx"]) if i % 2 else 0, take))
        left -= take
    return got


# ---------------------------------------------------------------------------
# the cache's format, in plain torch
# ---------------------------------------------------------------------------

MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _codes(y):
    """e2m1 codes of y, round to nearest even; magnitudes above 6 become 6."""
    a = y.abs()
    n = torch.zeros(y.shape, dtype=torch.uint8, device=y.device)
    for at, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        n += a >= at if up else a > at
    return n | (torch.signbit(y).to(torch.uint8) << 3)


def _pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _values(packed):
    """The values of packed codes, the last dimension twice as long."""
    t = torch.tensor(MAGNITUDES, device=packed.device)
    t = torch.cat([t, -t])
    pairs = torch.stack([t.repeat(16), t.repeat_interleave(16)], 1)            # of a byte: its low half's, its high half's
    return pairs[packed.int()].flatten(-2)


def _power(e8m0):
    """The value of e8m0 bytes above 0."""
    b = e8m0.int()
    return torch.where(b == 255, math.nan, (b << 23).view(torch.float32))


def _quantise_k(x):
    """x fp32 [...][D] -> packed codes [...][D/2], scale bytes [...][D/32]."""
    b = x.unflatten(-1, (-1, 32))
    m, e = torch.frexp(b.abs().amax(-1))
    e = torch.where(m > 0, e - 3 + (m >= 0.875), -100).clamp(min=-100)
    scale = (e + 127).to(torch.uint8)
    return _pack(_codes(b / _power(scale)[..., None]).flatten(-2)), scale


def _quantise_v(x):
    """x fp32 [...][D] -> codes [...][D], bf16 scales [...]."""
    s = (x.abs().amax(-1) / 6.0).clamp(min=2.0 ** -100).to(torch.bfloat16)
    return _codes(x / s.float()[..., None]), s


def _cache(pages, hk, page, d, gen):
    """A cache as the append leaves it, of pages that are full."""
    def normal(gain):
        x = torch.randn(pages, hk, page, d, generator=gen, device="cuda")
        return x.mul_(gain * torch.exp(0.5 * torch.randn(pages, hk, page, 1, generator=gen, device="cuda")))

    kc, ks = _quantise_k(normal(0.8))
    v, vs = _quantise_v(normal(0.5))
    v = _pack(v.unflatten(2, (-1, 16)).transpose(3, 4).contiguous())
    return kc, v, ks.transpose(2, 3).contiguous(), vs


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _frequencies(rot, yarn):
    """Rotary frequencies in 64 bits; with `yarn`, a 32,768-token model's scaled by 4 (Peng et al. 2023, section 3.4): slow
    frequencies divided by 4, fast ones kept, a ramp between. And the factor of the rotated elements."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 1e6 ** (-2.0 * i / rot)
    if not yarn:
        return f, 1.0
    turns = 32768 * f / (2 * math.pi)
    keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
    return f * keep + f / 4.0 * (1 - keep), 0.1 * math.log(4.0) + 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, bf16 = case["op"], torch.bfloat16
    hq, hk, d, page = case["hq"], case["hk"], case["d"], case["page"]
    lens = _lengths(case)
    ctx = torch.tensor([c for c, _ in lens], dtype=torch.int32)
    new = torch.tensor([n for _, n in lens], dtype=torch.int32)
    S, T = len(lens), int(new.sum())
    qsl = torch.cat([torch.zeros(1, dtype=torch.int64), new.long().cumsum(0)])
    # the pages of each request that the call reaches: all but for the update, those of the new tokens for it
    start = ctx // page if op == "update" else torch.zeros_like(ctx)
    held = (ctx + new + page - 1) // page - start
    n_pages = int(held.sum()) + (640 if op == "update" else 3)
    ids = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    cols = int(held.max())
    table = torch.full((S, cols), -1, dtype=torch.int32, device="cuda")
    table[(torch.arange(cols)[None] < held[:, None]).cuda()] = ids[: int(held.sum())]
    kc, vc, ks, vs = _cache(n_pages, hk, page, d, gen)
    s = {"op": op, "k_cache": kc, "v_cache": vc, "k_scale": ks, "v_scale": vs, "table": table, "qsl": qsl.to(torch.int32).cuda()}
    if op == "attention":
        s.update(seq=(ctx + new).cuda(), scale=d ** -0.5, causal=case["causal"], window=case["window"], longest=int((ctx + new).max()),
                 most_new=int(new.max()), q=torch.randn(T, hq, d, generator=gen, device="cuda").mul_(1.5).to(bf16),
                 o=torch.empty(T, hq, d, dtype=bf16, device="cuda"))
        return s
    s.update(first=(ctx - start * page).cuda(), k_out=torch.empty(T, hk, d, dtype=bf16, device="cuda"),
             v_out=torch.empty(T, hk, d, dtype=bf16, device="cuda"))
    if op == "read":
        return s
    # q, k and v are columns of the projection's output
    qkv = torch.randn(T, hq + 2 * hk, d, generator=gen, device="cuda")
    qkv *= torch.exp(0.7 * torch.randn(T, hq + 2 * hk, 1, generator=gen, device="cuda"))
    qkv = qkv.to(bf16)
    of = torch.repeat_interleave(torch.arange(S), new.long())
    pos = (ctx.long()[of] + torch.arange(T) - qsl[of]).cuda()
    slots = table[of.cuda(), pos // page - (ctx // page)[of].cuda()].long() * page + pos % page
    freq, rope_scale = _frequencies(case["rot"], case["yarn"])
    s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hk], v=qkv[:, hq + hk:], positions=pos.to(torch.int32), slots=slots, freq=freq.cuda(),
             rope_scale=rope_scale, interleaved=case["interleaved"], q_out=torch.empty(T, hq, d, dtype=bf16, device="cuda"))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_update(s):
    import gated_deltanet_token_amd as gdn
    gdn.gdn_rope_append_kv4(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["freq"], s["q_out"], s["k_cache"], s["v_cache"],
                            s["k_scale"], s["v_scale"], interleaved=s["interleaved"], rope_scale=s["rope_scale"])
    return [s["q_out"], *_own_read(s)]


def _own_read(s):
    import gated_deltanet_token_amd as gdn
    gdn.gdn_paged_read_kv4(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["first"], s["qsl"], s["k_out"],
                           s["v_out"])
    return [s["k_out"], s["v_out"]]


def _own_attention(s):
    import gated_deltanet_token_amd as gdn
    if "workspace" not in s:      # kept by the program, as its other buffers
        n = gdn.gdn_paged_attention_kv4_workspace_size(s["q"].shape[0], s["seq"].numel(), s["q"].shape[1], s["k_cache"].shape[1],
                                                       s["q"].shape[2], s["longest"])
        s["workspace"] = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    gdn.gdn_paged_attention_kv4(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["seq"], s["qsl"],
                                s["o"], s["longest"], scale=s["scale"], causal=s["causal"], window=s["window"],
                                workspace=s["workspace"])
    return s["o"]


_own = {"update": _own_update, "read": _own_read, "attention": _own_attention}


def _rotated(x, cos, sin, interleaved):
    """x in 64 bits [T][H][D], its first 2 * cos.shape[1] elements rotated."""
    n = cos.shape[1]
    r, rest = x[..., : 2 * n], x[..., 2 * n:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :n], r[..., n:])
    c, s = cos[:, None], sin[:, None]
    p, q = a * c - b * s, b * c + a * s
    r = torch.stack([p, q], -1).flatten(-2) if interleaved else torch.cat([p, q], -1)
    return torch.cat([r, rest], -1)


def _plain_update(s):
    angle = s["positions"].double()[:, None] * s["freq"][None]
    cos, sin = s["rope_scale"] * torch.cos(angle), s["rope_scale"] * torch.sin(angle)
    q = _rotated(s["q"].double(), cos, sin, s["interleaved"]).float().to(torch.bfloat16)
    k = _rotated(s["k"].double(), cos, sin, s["interleaved"]).float()
    page = s["v_scale"].shape[2]
    at, off = s["slots"] // page, s["slots"] % page
    s["k_cache"][at, :, off], s["k_scale"][at, :, :, off] = _quantise_k(k)
    codes, s["v_scale"][at, :, off] = _quantise_v(s["v"].float())
    # a value's codes share their bytes with a neighbouring token's: the touched pages are taken apart and put together again
    pages, of = torch.unique(at, return_inverse=True)
    v = s["v_cache"][pages]
    v = torch.stack([v & 15, v >> 4], -1).flatten(-2).transpose(3, 4)                     # [P][hk][page/16][16][D]
    v[of, :, off // 16, off % 16] = codes
    s["v_cache"][pages] = _pack(v.transpose(3, 4))
    return [q, *_plain_read(s)]


def _plain_read(s):
    page = s["v_scale"].shape[2]
    qsl = s["qsl"].long()
    t = torch.arange(s["k_out"].shape[0], device="cuda")
    of = torch.searchsorted(qsl[1:].contiguous(), t, right=True)
    j = s["first"].long()[of] + t - qsl[of]
    at, off = s["table"][of, j // page].long(), j % page
    k = _values(s["k_cache"][at, :, off]).unflatten(-1, (-1, 32)) * _power(s["k_scale"][at, :, :, off])[..., None]
    v = s["v_cache"][at, :, off // 16, :, off % 16 // 2]                                   # [T][hk][D]
    v = torch.where((off % 2 == 1)[:, None, None], v >> 4, v & 15)
    v = _values(v)[..., 0::2] * s["v_scale"][at, :, off].float()[..., None]
    return [k.flatten(-2).to(torch.bfloat16), v.to(torch.bfloat16)]


def _plain_attention(s):
    table, seq, qsl = s["table"].long(), s["seq"].long(), s["qsl"].long()
    S, (hk, page) = table.shape[0], s["v_scale"].shape[1:]
    T, hq, D = s["q"].shape
    G, L, N = hq // hk, table.shape[1] * page, s["most_new"]
    new = qsl[1:] - qsl[:-1]
    bt = table.clamp(min=0)
    k = _values(s["k_cache"][bt]).unflatten(-1, (-1, 32)) * _power(s["k_scale"][bt]).transpose(-1, -2)[..., None]
    k = k.flatten(-2).permute(0, 2, 4, 1, 3).reshape(S, hk, D, L)                          # from [S][P][hk][page][D]
    v = _values(s["v_cache"][bt]).transpose(-1, -2).flatten(3, 4) * s["v_scale"][bt].float()[..., None]
    v = v.transpose(1, 2).reshape(S, hk, L, D)                                             # from [S][P][hk][page][D]
    j, i = torch.arange(L, device="cuda"), torch.arange(N, device="cuda")
    live = (j < seq[:, None]) & (table >= 0).repeat_interleave(page, 1)                    # [S][L]
    v = torch.where(live[:, None, :, None], v, 0.0)
    # the requests' rows, padded to the longest: [S][hk][G N][D]
    row = (qsl[:-1, None] + i).clamp(max=T - 1)
    q = s["q"].float()[row].view(S, N, hk, G, D).permute(0, 2, 3, 1, 4).reshape(S, hk, G * N, D)
    x = torch.matmul(q, k).mul_(s["scale"]).view(S, hk, G, N, L)
    at = (seq - new)[:, None] + i                                                          # [S][N]
    keep = live[:, None, :].expand(S, N, L)
    if s["causal"]:
        keep = keep & (j <= at[..., None])
    if s["window"]:
        keep = keep & (j > at[..., None] - s["window"])
    x.masked_fill_(~keep[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = x.sum(-1)                                                                      # [S][hk][G][N]
    o = torch.matmul(x.view(S, hk, G * N, L), v).view(S, hk, G, N, D)
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    of = torch.searchsorted(qsl[1:].contiguous(), torch.arange(T, device="cuda"), right=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(S, N, hq, D)
    return o[of, torch.arange(T, device="cuda") - qsl[of]].to(torch.bfloat16)


_plain = {"update": _plain_update, "read": _plain_read, "attention": _plain_attention}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    lens, hq, hk, d = _lengths(case), case["hq"], case["hk"], case["d"]
    S, T = len(lens), sum(n for _, n in lens)
    stored = hk * (d + d // 32 + 2)                     # bytes of a token's codes and scales, k and v
    if case["op"] == "read":
        return {"bytes": T * (stored + 4 * hk * d) + 4 * sum(n // case["page"] + 1 for _, n in lens), "flops": 2 * T * hk * d}
    if case["op"] == "update":
        # q in and out, k and v in, codes and scales out, k and v out
        return {"bytes": T * (4 * hq * d + 8 * hk * d + stored + 12) + 4 * case["rot"],
                "flops": T * (3 * case["rot"] * (hq + hk) + 8 * hk * d)}
    keys, pairs = 0, 0
    for c, n in lens:
        L, w = c + n, case["window"]
        lo = max(0, c + 1 - w) if w else 0                               # the first key that some row sees
        keys += L - lo
        if case["causal"] and w:
            pairs += sum(min(w, p + 1) for p in range(c, L))
        elif case["causal"]:
            pairs += n * c + n * (n + 1) // 2
        elif w:
            pairs += sum(L - max(0, p + 1 - w) for p in range(c, L))
        else:
            pairs += n * L
    return {"bytes": stored * keys + 4 * T * hq * d + 4 * (keys // case["page"] + 3 * S), "flops": 4 * hq * d * pairs}


# ---------------------------------------------------------------------------
# the operators' definitions in 64 bits
# ---------------------------------------------------------------------------

def _e2m1(x):
    """x in 64 bits at the nearest of the format's values, ties to even: steps of 0.5 below 2, of 1 below 4, of 2 from there."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=1.0))) - 1)
    return (torch.round(x / step) * step).clamp(-6, 6)


def _exact_update(s):
    angle = s["positions"].double().outer(s["freq"])
    turn = s["rope_scale"] * torch.polar(torch.ones_like(angle), angle)
    n = s["freq"].numel()

    def rotate(x):
        x = x.double().clone()
        first = slice(0, 2 * n, 2) if s["interleaved"] else slice(0, n)
        second = slice(1, 2 * n, 2) if s["interleaved"] else slice(n, 2 * n)
        z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn[:, None]
        x[..., first], x[..., second] = z.real, z.imag
        return x

    k = rotate(s["k"]).float().double().reshape(*s["k"].shape[:2], -1, 32)
    top = k.abs().amax(-1, keepdim=True)
    unit = torch.exp2(torch.floor(torch.log2(top.clamp(min=1e-30))) - 2)
    unit = torch.where(top < 7 * unit, unit, 2 * unit)
    v = s["v"].double()
    sixth = (v.abs().amax(-1, keepdim=True) / 6).to(torch.bfloat16).double()
    return [rotate(s["q"]), (_e2m1(k / unit) * unit).flatten(-2), _e2m1(v / sixth) * sixth]


def _stored(s, ids, h):
    """Keys and values of head h of the pages `ids`, in order, in 64 bits: [tokens][D]."""
    of = torch.tensor([(1 - 2 * (c >> 3)) * MAGNITUDES[c & 7] for c in range(16)], dtype=torch.float64, device="cuda")
    kc, vc = s["k_cache"][ids, h].long(), s["v_cache"][ids, h].long()
    k = torch.empty(*kc.shape[:2], 2 * kc.shape[2], dtype=torch.float64, device="cuda")
    k[..., 0::2], k[..., 1::2] = of[kc % 16], of[kc // 16]
    power = torch.exp2(s["k_scale"][ids, h].double() - 127)                                # [n][D/32][page]
    k = k * power.transpose(1, 2).repeat_interleave(32, 2)
    v = torch.empty(*vc.shape[:3], 16, dtype=torch.float64, device="cuda")                 # [n][page/16][D][16]
    v[..., 0::2], v[..., 1::2] = of[vc % 16], of[vc // 16]
    v = v.permute(0, 1, 3, 2).reshape(*k.shape) * s["v_scale"][ids, h].double()[..., None]
    return k.flatten(0, 1), v.flatten(0, 1)


def _exact_read(s):
    hk, page = s["v_scale"].shape[1:]
    first, qsl = s["first"].tolist(), s["qsl"].tolist()
    k_out = torch.empty(s["k_out"].shape, dtype=torch.float64, device="cuda")
    v_out = torch.empty_like(k_out)
    for r, a in enumerate(first):
        lo, hi = qsl[r], qsl[r + 1]
        p = a // page
        ids = s["table"][r, p: (a + hi - lo - 1) // page + 1].long()
        for h in range(hk):
            k, v = _stored(s, ids, h)
            k_out[lo:hi, h], v_out[lo:hi, h] = k[a - p * page:][: hi - lo], v[a - p * page:][: hi - lo]
    return [k_out, v_out]


def _exact_attention(s):
    seq, qsl = s["seq"].tolist(), s["qsl"].tolist()
    hk, page = s["v_scale"].shape[1:]
    T, hq, D = s["q"].shape
    G = hq // hk
    o = torch.zeros(T, hq, D, dtype=torch.float64, device="cuda")
    for r, L in enumerate(seq):
        a, b = qsl[r], qsl[r + 1]
        ids = s["table"][r, : -(-L // page)].long()
        pos = torch.arange(L - (b - a), L, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")[None]
        seen = torch.ones(b - a, L, dtype=torch.bool, device="cuda")
        if s["causal"]:
            seen &= j <= pos
        if s["window"]:
            seen &= j > pos - s["window"]
        for h in range(hk):
            k, v = (x[:L] for x in _stored(s, ids, h))
            for g in range(h * G, h * G + G):
                w = (s["q"][a:b, g].double() @ k.T) * s["scale"]
                w = torch.softmax(w.masked_fill(~seen, -math.inf), -1)
                o[a:b, g] = torch.nan_to_num(w, nan=0.0) @ v
    return o


def exact(case, seed):
    s = prepare(case, seed)
    return {"update": _exact_update, "read": _exact_read, "attention": _exact_attention}[case["op"]](s)
