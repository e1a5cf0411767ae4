"""What the serving operators beside the Gated DeltaNet mixer cost, and what they compute.

Four operators of a hybrid model's engine step, each through its public entry point (``own``) or in plain torch:

  tables     gdn_build_step_tables: query_start_loc, sequence lengths, positions, cache slots, newly taken pages and conv
             descriptors of a step, from the requests' lengths
  append     gdn_rope_append_kv8: rotary positions on q and k, and the step's k and v written into the 8-bit paged cache
  attention  gdn_paged_attention_kv8: attention of the step's tokens over that cache
  head_norm, residual_norm
             gdn_gated_rms_norm (the norm of a mixer's heads with its output gate) and gdn_residual_rms_norm (norm after
             a block, gate, residual scale and sum, norm before the next block)

The cache holds e4m3 codes with an fp32 scale per (page, kv head): k_cache [pages][kv heads][page][head dim], v_cache
[pages][kv heads][head dim][page].
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
    return [
        # a decode step at concurrency 32 (1,024-token prompts, up to 128 new tokens): the smallest call, all latency
        {"name": "tables_decode_32", "op": "tables", "decodes": 32, "ctx_lo": 1024, "ctx_hi": 1151, "chunks": 0,
         "chunk_tokens": 0, "chunk_ctx": 0, "mix": 1, "page": 16, "cols": 96},
        # a large server's step: thousands of decoding requests and prompts being read in
        {"name": "tables_mixed_4096", "op": "tables", "decodes": 4000, "ctx_lo": 17, "ctx_hi": 16384, "chunks": 96,
         "chunk_tokens": 12288, "chunk_ctx": 8000, "mix": 2, "page": 16, "cols": 1100},
        # the decode step's new keys and values
        {"name": "append_decode_32", "op": "append", "decodes": 32, "ctx_lo": 1024, "ctx_hi": 1151, "chunks": 0,
         "chunk_tokens": 0, "chunk_ctx": 0, "mix": 1, **small, "rot": 64, "interleaved": False, "yarn": False},
        # a mixed step at the 2,048-token budget: 29 decode rows and three prompt chunks
        {"name": "append_mixed_2048", "op": "append", "decodes": 29, "ctx_lo": 1024, "ctx_hi": 1151, "chunks": 3,
         "chunk_tokens": 2019, "chunk_ctx": 700, "mix": 3, **small, "rot": 64, "interleaved": False, "yarn": False},
        # long prompts read in at once, whole heads rotated in the interleaved layout, scaled for long contexts
        {"name": "append_prefill_16384", "op": "append", "decodes": 0, "ctx_lo": 0, "ctx_hi": 0, "chunks": 8,
         "chunk_tokens": 16384, "chunk_ctx": 100000, "mix": 4, **wide, "rot": 128, "interleaved": True, "yarn": True},
        # the decode step's attention
        {"name": "attention_decode_32", "op": "attention", "decodes": 32, "ctx_lo": 1024, "ctx_hi": 1151, "chunks": 0,
         "chunk_tokens": 0, "chunk_ctx": 0, "mix": 1, **small, "causal": True, "window": 0},
        # a few requests with very long contexts of unlike lengths
        {"name": "attention_decode_long", "op": "attention", "decodes": 5, "ctx_lo": 40000, "ctx_hi": 131071, "chunks": 0,
         "chunk_tokens": 0, "chunk_ctx": 0, "mix": 5, **wide, "causal": True, "window": 0},
        # the mixed step's attention
        {"name": "attention_mixed_2048", "op": "attention", "decodes": 29, "ctx_lo": 1024, "ctx_hi": 1151, "chunks": 3,
         "chunk_tokens": 2019, "chunk_ctx": 700, "mix": 3, **small, "causal": True, "window": 0},
        # one long prompt
        {"name": "attention_prefill_8192", "op": "attention", "decodes": 0, "ctx_lo": 0, "ctx_hi": 0, "chunks": 1,
         "chunk_tokens": 8192, "chunk_ctx": 0, "mix": 6, **wide, "causal": True, "window": 0},
        # the mixer's output norm over a prefill step's 32 heads of 128
        {"name": "head_norm_2048", "op": "head_norm", "rows": 2048, "heads": 32, "d": 128, "gate": True},
        # between two blocks at decode
        {"name": "residual_norm_32", "op": "residual_norm", "rows": 32, "d": 2560, "post": False, "gate": False},
        # between two blocks over long prompts, with the norm after the block and its gate
        {"name": "residual_norm_16384", "op": "residual_norm", "rows": 16384, "d": 4096, "post": True, "gate": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("tables", "append", "attention", "attention", "head_norm", "residual_norm"))
    if op == "head_norm":
        d = rng.choice((32, 64, 128, 256))
        return {"op": op, "rows": _log(rng, 1, 4096), "heads": rng.choice((1, 4, 6, 16, 32)), "d": d, "gate": rng.random() < 0.7}
    if op == "residual_norm":
        return {"op": op, "rows": _log(rng, 1, 16384), "d": 8 * _log(rng, 8, 512), "post": rng.random() < 0.5,
                "gate": rng.random() < 0.5}
    hk = rng.choice((1, 2, 4, 8))
    c = {"op": op, "hq": hk * rng.choice((1, 2, 4, 5, 8) if hk < 8 else (1, 2, 4)), "hk": hk, "d": rng.choice((64, 128, 256)),
         "page": rng.choice((16, 32, 64)), "mix": rng.randrange(1 << 20)}
    if op == "tables":
        n = _log(rng, 1, 4000)
        chunks = rng.choice((0, _log(rng, 1, 64)))
        hi = _log(rng, 32, 16384)
        c = {"op": op, "decodes": n, "ctx_lo": rng.randrange(1, 32), "ctx_hi": hi, "chunks": chunks,
             "chunk_tokens": chunks and max(chunks, _log(rng, 64, 12288)), "chunk_ctx": rng.choice((0, hi)), "mix": c["mix"],
             "page": c["page"]}
        c["cols"] = -(-(hi + max(c["chunk_tokens"], 1) + 1) // c["page"])
        return c
    form = rng.choice(("decode", "decode", "mixed", "prefill"))
    c.update(decodes=0, ctx_lo=1, ctx_hi=1, chunks=0, chunk_tokens=0, chunk_ctx=0)
    if op == "append":
        if form != "prefill":
            c.update(decodes=_log(rng, 1, 200), ctx_hi=_log(rng, 16, 4096))
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
    """(context, new) tokens of each request: decode rows first."""
    r = random.Random(case["mix"])
    got = [(r.randint(case["ctx_lo"], max(case["ctx_lo"], case["ctx_hi"])), 1) for _ in range(case["decodes"])]
    n, left = case["chunks"], case["chunk_tokens"]
    for i in range(n):
        rest = n - 1 - i
        take = left if not rest else max(1, min(left - rest, int(r.uniform(0.5, 1.5) * left / (rest + 1))))
        got.append((r.randint(0, case["chunk_ctx"]) if i % 2 else 0, take))
        left -= take
    return got


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


def _quantised_cache(pages, hk, page, d, gen):
    """A cache as the append leaves it: e4m3 codes and a power-of-two scale per (page, kv head), k and v."""
    got = []
    for gain in (1.0, 0.5):
        x = torch.randn(pages, hk, page, d, generator=gen, device="cuda")
        x *= gain * torch.exp(0.5 * torch.randn(pages, hk, 1, 1, generator=gen, device="cuda"))
        m, e = torch.frexp(x.abs().amax(dim=(2, 3)))
        scale = torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875))
        got += [(x / scale[:, :, None, None]).to(torch.float8_e4m3fn), scale]
        del x
    k, ks, v, vs = got
    return k, v.view(torch.uint8).transpose(2, 3).contiguous().view(torch.float8_e4m3fn), ks, vs


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    bf16 = torch.bfloat16
    if op in ("head_norm", "residual_norm"):
        shape = (case["rows"], case["heads"], case["d"]) if op == "head_norm" else (case["rows"], case["d"])
        s = {"op": op, "eps": 1e-6, "x": torch.randn(shape, generator=gen, device="cuda").to(bf16),
             "weight": (0.2 * torch.randn(case["d"], generator=gen, device="cuda")).to(bf16), "gate": None, "post": None}
        if case["gate"]:
            s["gate"] = torch.randn(shape, generator=gen, device="cuda").to(bf16)
        s["y"] = torch.empty_like(s["x"])
        if op == "residual_norm":
            s["residual"] = (3 * torch.randn(shape, generator=gen, device="cuda")).to(bf16)
            s["new_residual"] = torch.empty_like(s["x"])
            s["alpha"] = 0.7
            if case["post"]:
                s["post"] = (0.2 * torch.randn(case["d"], generator=gen, device="cuda")).to(bf16)
        return s

    lens = _lengths(case)
    ctx = torch.tensor([c for c, _ in lens], dtype=torch.int32)
    new = torch.tensor([n for _, n in lens], dtype=torch.int32)
    S, T, page = len(lens), int(new.sum()), case["page"]
    have = (ctx + page - 1) // page
    want = (ctx + new + page - 1) // page
    if op == "tables":
        # each request's own pages are in its row; the others are free, in the order they came back
        cols = case["cols"]
        ids = torch.randperm(int(want.sum()) + 7, generator=gen, device="cuda").to(torch.int32)
        used = (torch.arange(cols)[None] < have[:, None]).cuda()
        n_used = int(have.sum())
        table = torch.full((S, cols), -1, dtype=torch.int32, device="cuda")
        table[used] = ids[:n_used]
        free = ids[n_used:].contiguous()
        i32 = {"dtype": torch.int32, "device": "cuda"}
        n_chunks = min(T, -(-T // 8) + S)
        return {"op": op, "page": page, "ctx": ctx.cuda(), "new": new.cuda(), "table": table, "free": free,
                "num_free": torch.tensor([free.numel()], **i32), "qsl": torch.zeros(S + 1, **i32), "seq": torch.zeros(S, **i32),
                "positions": torch.zeros(T, **i32), "slots": torch.zeros(T, dtype=torch.int64, device="cuda"),
                "chunks": torch.zeros(n_chunks, 2, **i32), "counts": torch.zeros(4, **i32)}

    hq, hk, d = case["hq"], case["hk"], case["d"]
    qsl = torch.cat([torch.zeros(1, dtype=torch.int64), new.long().cumsum(0)])
    # the pages of each request that the call reaches: all for the attention, those of the new tokens for the append
    start = torch.zeros_like(have) if op == "attention" else ctx // page
    held = want - start
    n_pages = int(held.sum()) + (3 if op == "attention" else 1280)
    ids = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    cols = int(held.max())
    table = torch.full((S, cols), -1, dtype=torch.int32, device="cuda")
    table[(torch.arange(cols)[None] < held[:, None]).cuda()] = ids[: int(held.sum())]
    kc, vc, ks, vs = _quantised_cache(n_pages, hk, page, d, gen)
    s = {"op": op, "k_cache": kc, "v_cache": vc, "k_scale": ks, "v_scale": vs}
    if op == "attention":
        s.update(table=table, seq=(ctx + new).cuda(), qsl=qsl.to(torch.int32).cuda(), scale=d ** -0.5, causal=case["causal"],
                 window=case["window"], longest=int((ctx + new).max()), most_new=int(new.max()),
                 q=torch.randn(T, hq, d, generator=gen, device="cuda").mul_(1.5).to(bf16),
                 o=torch.empty(T, hq, d, dtype=bf16, device="cuda"))
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


def _own_tables(s):
    import gated_deltanet_token_amd as gdn
    gdn.gdn_build_step_tables(s["ctx"], s["new"], s["free"], s["num_free"], s["table"], s["page"], s["qsl"], s["seq"],
                              s["positions"], s["slots"], s["counts"], chunks=s["chunks"])
    return [s["table"], s["qsl"], s["seq"], s["positions"], s["slots"], s["chunks"], s["counts"]]


def _own_append(s):
    import gated_deltanet_token_amd as gdn
    gdn.gdn_rope_append_kv8(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["freq"], s["q_out"], s["k_cache"], s["v_cache"],
                            s["k_scale"], s["v_scale"], interleaved=s["interleaved"], rope_scale=s["rope_scale"])
    return [s["q_out"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]]


def _own_attention(s):
    import gated_deltanet_token_amd as gdn
    if "workspace" not in s:      # kept by the program, as its other buffers
        n = gdn.gdn_paged_attention_kv8_workspace_size(s["q"].shape[0], s["seq"].numel(), s["q"].shape[1], s["k_cache"].shape[1],
                                                       s["q"].shape[2], s["longest"])
        s["workspace"] = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    gdn.gdn_paged_attention_kv8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["seq"], s["qsl"],
                                s["o"], s["longest"], scale=s["scale"], causal=s["causal"], window=s["window"],
                                workspace=s["workspace"])
    return s["o"]


def _own_head_norm(s):
    import gated_deltanet_token_amd as gdn
    gdn.gdn_gated_rms_norm(s["x"], s["weight"], s["y"], gate=s["gate"], eps=s["eps"], weight_offset=1.0)
    return s["y"]


def _own_residual_norm(s):
    import gated_deltanet_token_amd as gdn
    gdn.gdn_residual_rms_norm(s["x"], s["residual"], s["weight"], s["new_residual"], s["y"], post_weight=s["post"], gate=s["gate"],
                              residual_scale=s["alpha"], eps=s["eps"], weight_offset=1.0)
    return [s["new_residual"], s["y"]]


_own = {"tables": _own_tables, "append": _own_append, "attention": _own_attention, "head_norm": _own_head_norm,
        "residual_norm": _own_residual_norm}


def _plain_tables(s):
    page, table = s["page"], s["table"]
    ctx, new = s["ctx"].long(), s["new"].long()
    S, cols = table.shape
    seq = ctx + new
    have, want = (ctx + page - 1) // page, (seq + page - 1) // page
    n_chunk = (new + 7) // 8
    ends = new.cumsum(0)
    first_page, first_chunk = (want - have).cumsum(0) - (want - have), n_chunk.cumsum(0) - n_chunk
    qsl = torch.nn.functional.pad(ends, (1, 0))
    # taken pages come from the free list's end, request by request
    col = torch.arange(cols, device="cuda")[None]
    at = s["num_free"].long() - 1 - (first_page[:, None] + col - have[:, None])
    taken = (col >= have[:, None]) & (col < want[:, None])
    table = torch.where(taken, s["free"][at.clamp(0, s["free"].numel() - 1)], table)
    t = torch.arange(s["positions"].numel(), device="cuda")
    of = torch.searchsorted(ends, t, right=True)
    pos = ctx[of] + t - qsl[of]
    slots = table[of, pos // page].long() * page + pos % page
    c = torch.arange(s["chunks"].shape[0], device="cuda")
    of_c = torch.searchsorted(first_chunk + n_chunk, c, right=True)
    live = of_c < S
    of_c = of_c.clamp(max=S - 1)
    chunks = torch.stack([torch.where(live, of_c, -1), torch.where(live, c - first_chunk[of_c], 0)], 1)
    counts = torch.stack([ends[-1], n_chunk.sum(), (want - have).sum(), torch.zeros_like(ends[-1])])
    i32 = torch.int32
    return [table, qsl.to(i32), seq.to(i32), pos.to(i32), slots, chunks.to(i32), counts.to(i32)]


def _rotated(x, cos, sin, interleaved):
    """x in 64 bits [T][H][D], its first 2 * cos.shape[1] elements rotated."""
    n = cos.shape[1]
    r, rest = x[..., : 2 * n], x[..., 2 * n:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :n], r[..., n:])
    c, s = cos[:, None], sin[:, None]
    p, q = a * c - b * s, b * c + a * s
    r = torch.stack([p, q], -1).flatten(-2) if interleaved else torch.cat([p, q], -1)
    return torch.cat([r, rest], -1)


def _store(x, slots, cache, scale):
    """x [T][Hk][D] put into the cache's codes, uint8 [pages][Hk][page][D], at its slots, in place."""
    page, f8 = cache.shape[2], torch.float8_e4m3fn
    at, off = slots // page, slots % page
    pages, of = torch.unique(at, return_inverse=True)
    amax = torch.zeros(pages.numel(), x.shape[1], device="cuda").index_reduce_(0, of, x.abs().amax(-1), "amax")
    first = torch.full((pages.numel(),), page, device="cuda").index_reduce_(0, of, off, "amin")
    m, e = torch.frexp(amax)
    fit = torch.ldexp(torch.ones_like(m), torch.where(amax > 0, e - 9 + (m > 0.875), -100).clamp(min=-100))
    # a page that holds tokens already keeps its scale unless the new ones need a larger
    old, codes = scale[pages], cache[pages]
    now = torch.where((first > 0)[:, None], torch.maximum(old, fit), fit)
    kept = (codes.view(f8).float() * (old / now)[:, :, None, None]).to(f8).view(torch.uint8)
    codes = torch.where((torch.arange(page, device="cuda") < first[:, None])[:, None, :, None], kept, codes)
    codes[of, :, off] = (x / now[of][..., None]).to(f8).view(torch.uint8)
    cache[pages], scale[pages] = codes, now


def _plain_append(s):
    angle = s["positions"].double()[:, None] * s["freq"][None]
    cos, sin = s["rope_scale"] * torch.cos(angle), s["rope_scale"] * torch.sin(angle)
    q = _rotated(s["q"].double(), cos, sin, s["interleaved"]).float().to(torch.bfloat16)
    k = _rotated(s["k"].double(), cos, sin, s["interleaved"]).float()
    _store(k, s["slots"], s["k_cache"].view(torch.uint8), s["k_scale"])
    _store(s["v"].float(), s["slots"], s["v_cache"].view(torch.uint8).transpose(2, 3), s["v_scale"])
    return [q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]]


def _plain_attention(s):
    table, seq, qsl = s["table"].long(), s["seq"].long(), s["qsl"].long()
    S, hk, page, D = table.shape[0], *s["k_cache"].shape[1:]
    T, hq, _ = s["q"].shape
    G, L, N = hq // hk, table.shape[1] * page, s["most_new"]
    new = qsl[1:] - qsl[:-1]
    bt = table.clamp(min=0)
    f8 = torch.float8_e4m3fn
    k = s["k_cache"].view(torch.uint8)[bt].view(f8).float() * s["k_scale"][bt][..., None, None]       # [S][P][hk][page][D]
    k = k.permute(0, 2, 4, 1, 3).reshape(S, hk, D, L)
    v = s["v_cache"].view(torch.uint8)[bt].view(f8).float() * s["v_scale"][bt][..., None, None]       # [S][P][hk][D][page]
    v = v.permute(0, 2, 1, 4, 3).reshape(S, hk, L, D)
    j, i = torch.arange(L, device="cuda"), torch.arange(N, device="cuda")
    live = (j < seq[:, None]) & (table >= 0).repeat_interleave(page, 1)                                # [S][L]
    v = torch.where(live[:, None, :, None], v, 0.0)
    # the requests' rows, padded to the longest: [S][hk][G N][D]
    row = (qsl[:-1, None] + i).clamp(max=T - 1)
    q = s["q"].float()[row].view(S, N, hk, G, D).permute(0, 2, 3, 1, 4).reshape(S, hk, G * N, D)
    x = torch.matmul(q, k).mul_(s["scale"]).view(S, hk, G, N, L)
    at = (seq - new)[:, None] + i                                                                      # [S][N]
    keep = live[:, None, :].expand(S, N, L)
    if s["causal"]:
        keep = keep & (j <= at[..., None])
    if s["window"]:
        keep = keep & (j > at[..., None] - s["window"])
    x.masked_fill_(~keep[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = x.sum(-1)                                                                                  # [S][hk][G][N]
    o = torch.matmul(x.view(S, hk, G * N, L), v).view(S, hk, G, N, D)
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    of = torch.searchsorted(qsl[1:].contiguous(), torch.arange(T, device="cuda"), right=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(S, N, hq, D)
    return o[of, torch.arange(T, device="cuda") - qsl[of]].to(torch.bfloat16)


def _rms(x, weight, eps):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * (1.0 + weight.float())


def _plain_head_norm(s):
    y = _rms(s["x"].float(), s["weight"], s["eps"])
    if s["gate"] is not None:
        z = s["gate"].float()
        y = y * (z / (1.0 + torch.exp(-z)))
    return y.to(torch.bfloat16)


def _plain_residual_norm(s):
    u = s["x"].float()
    if s["post"] is not None:
        u = _rms(u, s["post"], s["eps"])
    if s["gate"] is not None:
        u = u / (1.0 + torch.exp(-s["gate"].float()))
    h = s["residual"].float() + s["alpha"] * u
    return [h.to(torch.bfloat16), _rms(h, s["weight"], s["eps"]).to(torch.bfloat16)]


_plain = {"tables": _plain_tables, "append": _plain_append, "attention": _plain_attention, "head_norm": _plain_head_norm,
          "residual_norm": _plain_residual_norm}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "head_norm":
        n = case["rows"] * case["heads"] * case["d"]
        return {"bytes": 2 * n * (3 if case["gate"] else 2) + 2 * case["d"], "flops": n * (9 if case["gate"] else 5)}
    if op == "residual_norm":
        n = case["rows"] * case["d"]
        return {"bytes": 2 * n * (5 if case["gate"] else 4) + 4 * case["d"], "flops": n * (7 + 5 * case["post"] + 4 * case["gate"])}
    lens, page = _lengths(case), case["page"]
    S, T = len(lens), sum(n for _, n in lens)
    taken = sum(-(-(c + n) // page) - -(-c // page) for c, n in lens)
    if op == "tables":
        # lengths in; query_start_loc, lengths, positions, slots, descriptors and counts out; taken pages read and written;
        # the page of each request's last, partly filled one read
        return {"bytes": 8 * S + 4 * (S + 1) + 4 * S + 12 * T + 8 * min(T, -(-T // 8) + S) + 8 * taken + 4 * S + 16, "flops": 10 * T}
    hq, hk, d = case["hq"], case["hk"], case["d"]
    if op == "append":
        # q in and out, k and v in, their codes out, a scale read and written per (page, head)
        touched = sum(-(-(c + n) // page) - c // page for c, n in lens)
        return {"bytes": T * d * (4 * hq + 6 * hk) + 12 * T + 4 * case["rot"] + 16 * touched * hk,
                "flops": T * (3 * case["rot"] * (hq + hk) + 6 * hk * d)}
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
    return {"bytes": 2 * hk * d * keys + 4 * T * hq * d + 12 * hk * (keys // page + S), "flops": 4 * hq * d * pairs}


# ---------------------------------------------------------------------------
# the operators' definitions in 64 bits
# ---------------------------------------------------------------------------

def _e4m3(x):
    """x in 64 bits at the nearest value of 4 exponent and 3 mantissa bits (ties to even; largest 448, smallest 2^-9)."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_append(s):
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

    out = [rotate(s["q"])]
    slots = s["slots"].tolist()
    for x, cache, scale in ((rotate(s["k"]).float().double(), s["k_cache"], s["k_scale"]),
                            (s["v"].double(), s["v_cache"].view(torch.uint8).transpose(2, 3).view(torch.float8_e4m3fn), s["v_scale"])):
        page = cache.shape[2]
        cache, scale = cache.double(), scale.double()
        t = 0
        while t < len(slots):                       # one page's new tokens at a time
            p, off = divmod(slots[t], page)
            n_new = 1
            while t + n_new < len(slots) and off + n_new < page and slots[t + n_new] == slots[t] + n_new:
                n_new += 1
            y = x[t:t + n_new].transpose(0, 1)                                # [Hk][n][D]
            need = torch.exp2(torch.ceil(torch.log2(y.abs().amax(dim=(1, 2)) / 448)).clamp(min=-100))
            now = torch.maximum(need, scale[p]) if off else need
            cache[p, :, :off] = _e4m3(cache[p, :, :off] * (scale[p] / now)[:, None, None])
            cache[p, :, off:off + n_new] = _e4m3(y / now[:, None, None])
            scale[p] = now
            t += n_new
        out += [cache, scale]
    q, kc, ks, vc, vs = out
    return [q, kc, vc.transpose(2, 3).contiguous(), ks, vs]


def _exact_attention(s):
    seq, qsl, table = s["seq"].tolist(), s["qsl"].tolist(), s["table"]
    hk, page, D = s["k_cache"].shape[1:]
    T, hq, _ = s["q"].shape
    G = hq // hk
    o = torch.zeros(T, hq, D, dtype=torch.float64, device="cuda")
    for r, L in enumerate(seq):
        a, b = qsl[r], qsl[r + 1]
        ids = table[r, : -(-L // page)].long()
        pos = torch.arange(L - (b - a), L, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")[None]
        seen = torch.ones(b - a, L, dtype=torch.bool, device="cuda")
        if s["causal"]:
            seen &= j <= pos
        if s["window"]:
            seen &= j > pos - s["window"]
        for h in range(hk):
            k = (s["k_cache"].view(torch.uint8)[ids, h].view(torch.float8_e4m3fn).double() * s["k_scale"][ids, h].double()[:, None, None])
            v = (s["v_cache"].view(torch.uint8)[ids, h].view(torch.float8_e4m3fn).double() * s["v_scale"][ids, h].double()[:, None, None])
            k, v = k.reshape(-1, D)[:L], v.transpose(1, 2).reshape(-1, D)[:L]
            for g in range(h * G, h * G + G):
                w = (s["q"][a:b, g].double() @ k.T) * s["scale"]
                w = torch.softmax(w.masked_fill(~seen, -math.inf), -1)
                o[a:b, g] = torch.nan_to_num(w, nan=0.0) @ v
    return o


def _exact_norm(x, weight, eps):
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + eps) * (weight.double() + 1)


def exact(case, seed):
    if case["op"] == "tables":
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "attention":
        return _exact_attention(s)
    x = s["x"].double()
    z = s["gate"].double() if s["gate"] is not None else None
    if case["op"] == "head_norm":
        y = _exact_norm(x, s["weight"], s["eps"])
        return y if z is None else y * z * torch.sigmoid(z)
    if s["post"] is not None:
        x = _exact_norm(x, s["post"], s["eps"])
    if z is not None:
        x = x * torch.sigmoid(z)
    h = s["residual"].double() + s["alpha"] * x
    return [h, _exact_norm(h, s["weight"], s["eps"])]
