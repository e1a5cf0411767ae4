"""GPU checks of gdn_paged_attention_kv4 against the formula in 64 bits.

Bound per element: 2^-8 |o| for the final rounding to bf16, and for the weights'
own rounding to bf16 2^-8 sum_j w_j |v_j|.  Scores off by at most e change weights,
numerator and sum together, by at most 2 e of themselves, and o by 2 e sum_j w_j |v_j|:
e is what q's three parts leave out (split_error, from their definition and the largest
codes of the cache), and for sums and exponentials in fp32 2^-11 sum_j w_j |v_j| at the score
sizes used here (|x| below 60)."""
import numpy as np
import pytest
import torch

import gated_deltanet_token_amd as gdn
import kv4_ref as kv4
import serving_ref as ref
from test_gpu_serving_attention import DECODE, HEADS, MIXED, cuda

pytestmark = pytest.mark.gpu


class Case:
    """A batch of (kv length, new tokens) requests over a random cache."""

    def __init__(self, seed, lens, hq, hk, d, page, spare_cols=1, spread=1.0):
        r = self.r = np.random.default_rng(seed)
        S = len(lens)
        self.seq = np.array([L for L, _ in lens], np.int32)
        self.qsl = np.concatenate([[0], np.cumsum([n for _, n in lens])]).astype(np.int32)
        T = int(self.qsl[-1])
        need = -(-np.maximum(self.seq, 0) // page)
        pages = int(need.sum()) + 3
        ids = r.permutation(pages)
        self.table = np.full((S, int(need.max(initial=0)) + spare_cols), -1, np.int32)
        at = 0
        for s in range(S):
            self.table[s, :need[s]] = ids[at:at + need[s]]
            at += need[s]
        shape = (pages, hk, page, d)
        self.kq, self.ks = kv4.quantise_k(r.standard_normal(shape) * np.exp(0.5 * r.standard_normal((pages, hk, page, 1))))
        self.vq, self.vs = kv4.quantise_v(r.standard_normal(shape) * np.exp(2 * r.standard_normal((pages, hk, page, 1))))
        self.q = cuda((spread * r.standard_normal((T, hq, d))).astype(np.float32), torch.bfloat16)
        self.scale = d ** -0.5
        # what lies past a request's end is anybody's: scales of NaN
        for s in range(S):
            L = max(int(self.seq[s]), 0)
            if L % page:
                p = self.table[s, L // page]
                self.ks[p, :, L % page:], self.vs[p, :, L % page:] = 255, np.nan

    def gpu(self):
        t = lambda x: torch.tensor(x, device="cuda")                                       # noqa: E731
        return dict(k_cache=t(kv4.pack_k(self.kq)), v_cache=t(kv4.pack_v(self.vq)), k_scale=t(kv4.pack_k_scale(self.ks)),
                    v_scale=t(self.vs.astype(np.float32)).to(torch.bfloat16), block_table=cuda(self.table, torch.int32),
                    seq_lens=cuda(self.seq, torch.int32), query_start_loc=cuda(self.qsl, torch.int32))

    def longest(self):
        return max(int(self.seq.max(initial=1)), 1)

    def values(self):
        """k [pages][hk][page][D], v [pages][hk][D][page]"""
        return kv4.key_values(self.kq, self.ks), kv4.value_values(self.vq, self.vs).swapaxes(2, 3)

    def want(self, **kw):
        k, v = self.values()
        one = np.ones(k.shape[:2])
        return ref.attention(ref.values(self.q), k, v, one, one, self.table, self.seq, self.qsl, self.scale, **kw)

    def split_error(self):
        """The most that q's parts can change a score by."""
        q = ref.values(self.q).reshape(*self.q.shape[:2], -1, 32)
        k = np.abs(kv4.key_values(self.kq, np.where(self.ks >= 250, 0, self.ks)))           # (those are not seen)
        k = k.reshape(*self.kq.shape[:3], -1, 32)
        most = np.repeat(k.max((0, 2)), self.q.shape[1] // k.shape[1], 0)                  # [hq][blocks][32]
        return abs(self.scale) * (np.abs(kv4.split(q) - q) * most).sum((-1, -2)).max(initial=0.0)

    def run(self, longest=None, q=None, **kw):
        q = self.q if q is None else q
        o = torch.full(q.shape, 77.0, dtype=torch.bfloat16, device="cuda")
        gdn.gdn_paged_attention_kv4(q, o=o, max_seq_len=longest or self.longest(), scale=self.scale, **self.gpu(), **kw)
        torch.cuda.synchronize()
        return o

    def near(self, o, want, mag):
        got = ref.values(o)
        owned = ~(mag < 0).all(-1)
        assert (got[~owned] == 77.0).all()
        assert np.array_equal(np.isnan(got[owned]), np.isnan(want[owned]))
        err = np.abs(got - want)[owned]
        bound = (np.abs(want) * 2.0 ** -8 + mag * (2.0 ** -8 + 2.0 ** -11 + 2 * self.split_error()) + 1e-30)[owned]
        fine = ~np.isnan(want[owned])
        assert (err[fine] <= bound[fine]).all(), "%.3g of the bound" % (err[fine] / bound[fine]).max()

    def check(self, longest=None, most=2.0 ** -8, **kw):
        assert self.split_error() < most
        o = self.run(longest, **kw)
        self.near(o, *self.want(**kw))
        return o


@pytest.mark.parametrize("d,page", [(64, 16), (64, 64), (128, 16), (128, 32), (256, 16), (256, 64)])
@pytest.mark.parametrize("hq,hk", HEADS)
def test_decode(d, page, hq, hk):
    Case(d + page + hq, DECODE, hq, hk, d, page).check()


@pytest.mark.parametrize("d,page", [(64, 32), (128, 16), (128, 64), (256, 32)])
@pytest.mark.parametrize("hq,hk", HEADS)
def test_mixed(d, page, hq, hk):
    Case(d + page + hq, MIXED, hq, hk, d, page).check()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 16), (True, 33), (True, 100), (False, 40), (False, 1000)])
def test_masks(d, causal, window):
    Case(d + window, MIXED + DECODE[:5], 8, 2, d, 16).check(causal=causal, window=window)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompts(d):
    Case(3, [(257, 257), (500, 300), (128, 128), (129, 127)], 4, 2, d, 16, spread=3.0).check()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [17, 31, 32, 33, 48, 63, 64, 65, 96, 127, 129])
def test_rows_about_a_tile(d, new):
    """Two rows per token and kv head: 33 rows and more are a large request's, of whole and
    of broken tiles."""
    Case(new, [(new + 70, new), (5, 1), (new, new)], 4, 2, d, 16).check()


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("window", [100, 1024, 1025])
def test_windows_over_long_requests(d, window):
    """A window of one part's keys or fewer, wherever it lies: few rows are not split."""
    c = Case(31, [(9000, 1), (4097, 1), (1500, 1), (3, 1)], 4, 1, d, 16)
    for longest in (None, 1, 100, 1023, 1024, 2 ** 31 - 1):
        c.check(longest, window=window)
    Case(32, [(9000, 1), (4097, 3), (5000, 90), (3, 1)], 4, 1, d, 16).check(window=window)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_long_decode_in_parts(d):
    """Few rows over long contexts: the work is split along the keys and joined."""
    c = Case(4, [(9000, 1), (4097, 1), (3, 1)], 4, 1, d, 32, spread=4.0)
    c.check()
    c.check(window=5000)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens", [[(640, 40)], [(1300, 300)], [(5000, 64)], [(3000, 100), (700, 50), (40, 40)],
                                  [(5000, 1), (4100, 2), (3000, 60)], [(2500, 1)] * 3 + [(2500, 3), (5, 1), (9000, 33), (0, 0)]])
def test_chunks_and_small_requests_in_parts(d, lens):
    Case(5, lens, 4, 2, d, 16).check()


@pytest.mark.parametrize("n", [1, 3])
def test_max_seq_len_is_only_a_hint(n):
    c = Case(5, [(5000, n), (100, n)], 8, 2, 128, 16)
    want = c.want()
    for longest in (1, 100, 4999, 5000, 2 ** 31 - 1):
        c.near(c.run(longest), *want)


def test_rows_without_keys_are_zero():
    """More new tokens than keys, empty requests with tokens, lengths below zero."""
    c = Case(6, [(3, 10), (0, 4), (-7, 2), (20, 40)], 4, 2, 128, 16)
    o = c.check()
    assert (o[:7] == 0).all() and (o[10:16] == 0).all() and (o[16:36] == 0).all()
    c.check(causal=False)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_missing_pages_are_not_seen(d):
    c = Case(7, [(100, 1), (90, 30), (40, 1), (400, 2)], 4, 2, d, 16)
    c.table[0, 2], c.table[1, 0], c.table[1, 4], c.table[3, 11] = -1, 10 ** 6, -1, -2 ** 31
    c.table[2, :] = -1
    o = c.check()
    assert (o[31] == 0).all()
    c.check(causal=False)


def test_length_past_the_row_is_cut():
    c = Case(8, [(100, 1), (100, 30)], 4, 2, 64, 16, spare_cols=0)
    c.table = np.ascontiguousarray(c.table[:, :4])
    c.check()


@pytest.mark.parametrize("d,hq,hk", [(64, 4, 2), (128, 16, 1), (256, 8, 4)])
def test_bad_scales_reach_only_the_rows_that_see_them(d, hq, hk):
    """Scales of NaN of a key's block or a value: rows before it keep their results, rows after it are NaN."""
    page = 16
    c = Case(9, [(90, 90), (50, 1), (130, 70)], hq, hk, d, page)
    c.vs[c.table[0, 3], 0, 7] = np.nan          # request 0, key 55
    c.ks[c.table[2, 6], 0, 4, 1] = 255          # request 2, key 100: one block
    want, mag = c.want()
    got = ref.values(c.run())
    G = hq // hk
    assert np.isnan(got[55:90, :G]).all() and not np.isnan(got[:55]).any() and not np.isnan(got[90]).any()
    assert np.isnan(got[131:, :G]).all() and not np.isnan(got[91:131]).any() and not np.isnan(got[:, G:]).any()
    c.near(c.run(), want, mag)
    # NaN and infinite scales on pages that nobody's mask reaches
    c = Case(10, [(64, 1), (64, 64)], hq, hk, d, page)
    c.ks[c.table[0, 0]], c.vs[c.table[0, 0]] = 255, np.inf
    c.ks[c.table[0, 1]], c.vs[c.table[0, 1]] = 254, np.nan
    c.check(window=20)


def test_bad_queries_stay_in_their_rows():
    c = Case(11, MIXED, 8, 2, 128, 16)
    want, mag = c.want()
    q = c.q.clone()
    q[5, 3, 7], q[40, 0, 0], q[70, 7, 100] = float("nan"), float("inf"), float("-inf")
    got = c.run(q=q)
    for t, h in ((5, 3), (40, 0), (70, 7)):
        assert torch.isnan(got[t, h]).all()
        got[t, h] = torch.tensor(want[t, h]).to(got)
    c.near(got, want, mag)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_queries_of_uneven_size(d):
    """One element of a row hundreds of times the others, and tiny ones: q's three parts keep them."""
    c = Case(12, [(300, 20), (80, 1)], 4, 2, d, 16, spread=0.02)
    c.q[:, :, 5] *= 100
    c.check()
    c.q.mul_(2.0 ** -90)
    c.scale *= 2.0 ** 90
    c.check()
    c.q.zero_()
    c.check()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 3, 40], ids=["decode", "small", "large"])
def test_small_elements_beside_a_large_one(d, new):
    """Two keys: one without score, and one that meets a single element of q, 2^-level of
    its block's largest, with a score of -4 and a value of 1: o = e^x / (1 + e^x) follows that
    element.  Its weight is rounded once, and o; q's parts hold the element exactly down to
    level 7, and within 2^-15 of the largest from there on."""
    S = 70
    c = Case(13, [(2, new)] * S, 1, 1, d, 16)
    r, at = c.r, c.table[:, 0]
    level = np.arange(S) % 14
    small = (1 + r.integers(0, 128, S) / 128) * 2.0 ** -level
    e = r.integers(1, 32, S) + 32 * r.integers(0, d // 32, S)
    q = np.zeros((S, d))
    q[:, ::32] = 1.9921875 * r.choice([-1, 1], (S, d // 32))
    q[np.arange(S), e] = small
    c.q = cuda(np.repeat(q, new, 0)[:, None], torch.bfloat16)
    assert np.array_equal(ref.values(c.q)[::new, 0], q)
    c.kq[...], c.vq[...], c.vs[...], c.scale = 0, 0, 1.0, 1.0
    up = np.round(np.log2(4 / small)).astype(int)              # scores from -2.8 to -5.7
    c.ks[at] = (127 + up)[:, None, None, None]
    c.kq[at, 0, 1, e] = 10                                     # -1
    c.vq[at, 0, 1] = 2                                         # 1
    x = -small * 2.0 ** up
    want = np.repeat(np.exp(x) / (1 + np.exp(x)), new)
    off = np.where(level > 7, 2.0 ** -15 * 1.9921875 / small, 0.0) * np.abs(x)
    bound = want * np.repeat(2 * 2.0 ** -8 + 2.0 ** -15 + 1.01 * off, new)
    err = np.abs(ref.values(c.run(causal=False))[:, 0] - want[:, None]).max(-1)
    assert (err <= bound).all(), (err / bound).max()


@pytest.mark.parametrize("d", [64, 256])
def test_value_scales_far_apart(d):
    c = Case(14, [(200, 1), (200, 60)], 4, 1, d, 16)
    c.vs[:, :, ::2] *= 2.0 ** 40
    c.vs[:, :, 1::2] *= 2.0 ** -60
    c.check()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_value_scales_over_their_whole_range(d):
    """Every token's scale another one from 2^-100 to 2^100, some zero or negative: none passes
    fp32's end in a weight, none's rounding reaches another row."""
    c = Case(19, [(300, 70), (90, 90), (500, 1), (64, 40)], 8, 2, d, 16, spread=2.0)
    c.vs = kv4.bf16(2.0 ** c.r.integers(-100, 101, c.vs.shape) * c.r.uniform(1, 2, c.vs.shape))
    c.vs[:, :, ::7] = 0
    c.vs[:, :, 1::5] *= -1
    c.check()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_key_scales_over_a_wide_range(d):
    """A key's blocks from 2^-100 to 2^30, q small where they are large."""
    c = Case(20, [(300, 70), (500, 1)], 4, 2, d, 16)
    x = c.r.integers(-100, 31, (1, 2, 1, d // 32))
    c.ks = np.broadcast_to(x + 127, c.ks.shape).astype(np.uint8).copy()
    up = torch.tensor(np.repeat(2.0 ** -x[0, :, 0].astype(np.float64), 32, -1), device="cuda").repeat_interleave(2, 0)
    c.q = (c.q.double() * up).to(torch.bfloat16)
    c.check()


def test_large_scores():
    """One key dominates; fully negative rows; the running maximum moves by hundreds."""
    c = Case(15, [(500, 3), (100, 100)], 4, 2, 64, 16, spread=1.0)
    c.scale = 0.9
    c.check()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("step", [1, 8, 9, 200])
def test_scores_that_rise_or_fall_with_the_key(d, step):
    """The running maximum moves by `step` powers of two per 16 keys, up in one kv head and
    down in the other: sums follow it at once, late, or not at all."""
    c = Case(20, [(200, 100), (330, 1), (150, 33)], 4, 2, d, 16, spread=0.0)
    c.q[...] = 0
    c.kq[...] = 0
    c.ks[...] = 127
    # base-4 digits of the number, digit i in element i, met by 4^i of q
    c.q[:, :, :8] = torch.tensor(4.0 ** np.arange(8), device="cuda").to(torch.bfloat16)
    c.scale = np.log(2.0)
    for s in range(len(c.seq)):
        for i in range(-(-int(c.seq[s]) // 16)):
            for h, n in enumerate((step * (i + 1), step * (40 - i))):
                digits = np.array([n >> 2 * b & 3 for b in range(8)])
                c.kq[c.table[s, i], h, :, :8] = np.array([0, 2, 4, 5])[digits]
    c.check()


@pytest.mark.parametrize("scale", [-0.125, 0.0, 1e-30, -3.0])
def test_scales_of_any_sign(scale):
    for d in (64, 128, 256):
        c = Case(21, [(100, 40), (70, 1)], 4, 2, d, 16, spread=0.5)
        c.scale = scale
        c.check()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 3, 40], ids=["decode", "small", "large"])
def test_light_keys_beside_heavy_ones(d, new):
    """Heavy keys whose values are zero: what the light ones hold is there to 2^-8 of it."""
    c = Case(22, [(700, new)], 2, 1, d, 16, spread=0.0)
    c.q[:, :, 0] = 16.0
    c.kq[:, :, :, 0] = 0
    c.ks[...] = 127
    c.scale = 1.0
    for i, p in enumerate(c.table[0, :44]):
        c.kq[p, 0, ::5, 0] = 2                    # these weigh e^16 times the others
        c.vq[p, 0, ::5] = 0
    assert c.split_error() == 0.0
    c.check()


def test_strided_operands_and_unowned_rows():
    c = Case(16, MIXED, 8, 2, 128, 16)
    T = c.q.shape[0]
    wide = torch.full((T + 9, 14, 128), 77.0, dtype=torch.bfloat16, device="cuda")
    qv, ov = wide[:, :8], torch.full((T + 9, 10, 128), 77.0, dtype=torch.bfloat16, device="cuda")
    qv[:T] = c.q
    g = c.gpu()
    bt = torch.full((len(MIXED), c.table.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    bt[:, :c.table.shape[1]] = g["block_table"]
    g["block_table"] = bt[:, :c.table.shape[1]]
    gdn.gdn_paged_attention_kv4(qv, o=ov[:, 1:9], max_seq_len=300, scale=c.scale, **g)
    torch.cuda.synchronize()
    c.near(ov[:T, 1:9], *c.want())
    assert (ov[T:] == 77).all() and (ov[:, 0] == 77).all() and (ov[:, 9] == 77).all()


def test_malformed_query_start_loc_stays_inside():
    c = Case(17, [(50, 10), (60, 10), (70, 10)], 4, 2, 64, 16)
    c.qsl = np.array([0, 25, 12, 900], np.int32)         # a decreasing and a far bound
    c.run()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens", [[(100, 1), (70, 1), (50, 1)], [(100, 1), (90, 3), (200, 60), (40, 1)]], ids=["decode", "mixed"])
@pytest.mark.parametrize("window,short", [(1, 0), (447, 64), (100, 500), (5000, 64)])
def test_windows_past_the_row(d, lens, window, short):
    """Requests longer than their row of the block table, by a little or up to 2^31 - 1."""
    c = Case(23, lens, 4, 2, d, 16, spare_cols=0)
    c.seq = c.seq + short
    c.check(window=window)
    c.seq[0] = 2 ** 31 - 1
    c.check(longest=200, window=window)


@pytest.mark.parametrize("d,hq,hk", [(64, 4, 2), (128, 40, 1), (256, 8, 4)])
@pytest.mark.parametrize("slots", [129, 130, 131, 700])
def test_prompts_among_empty_slots(d, hq, hk, slots):
    """130 tokens in a batch padded with requests that have none."""
    lens = [(0, 0)] * slots
    lens[1], lens[slots // 2], lens[slots - 1] = (100, 60), (90, 69), (33, 1)
    Case(24, lens, hq, hk, d, 16).check()


@pytest.mark.parametrize("hq,hk,d", [(40, 1, 64), (80, 2, 128), (40, 1, 256), (160, 1, 64), (160, 1, 128), (160, 1, 256)])
def test_groups_of_many_heads(hq, hk, d):
    Case(25, [(300, 1), (70, 3), (90, 20), (1, 1)], hq, hk, d, 16).check()
    Case(26, [(300, 1), (70, 1)], hq, hk, d, 32).check()


def test_more_requests_than_a_wave():
    r = np.random.default_rng(18)
    lens = [(int(r.integers(1, 60)), int(r.integers(0, 3))) for _ in range(150)]
    lens = [(max(L, n), n) for L, n in lens]
    Case(18, lens, 4, 2, 64, 16).check()
    Case(19, [(int(r.integers(1, 60)), 1) for _ in range(300)], 4, 2, 64, 16).check()


@pytest.mark.parametrize("d,hk", [(64, 8), (128, 5), (256, 4)])
@pytest.mark.parametrize("S", [257, 1024, 1025])
def test_many_requests_of_unlike_lengths(d, hk, S):
    """Over 1,024 (request, kv head) pairs, taken longest first up to 1,024 requests: empty ones,
    some with several tokens, equal lengths and one far longer than the others among them."""
    r = np.random.default_rng(S + d)
    n = np.ones(S, int)
    n[r.permutation(S)[:S // 4]] = 0
    n[r.permutation(np.flatnonzero(n == 0))[:3]] = (2, 7, 20)
    L = np.where(r.random(S) < 0.3, 20, r.integers(0, 70, S))
    L[r.integers(0, S)] = 700
    lens = [(max(int(a), int(b)) if r.random() < 0.9 else int(a), int(b)) for a, b in zip(L, n)]
    if sum(n) * hk <= 1024:
        hk = -(-1025 // int(sum(n)))
    c = Case(S, lens, hk, hk, d, 16)
    assert c.qsl[-1] <= S and c.qsl[-1] * hk > 1024
    c.check()
    if S == 257:
        c.check(longest=30)
        c.check(window=9)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_long_parts(d):
    """Parts of 2,048 keys and more, joined."""
    Case(27, [(9000, 1)] * 2 + [(20, 1), (30000, 1)] + [(7000, 1)] * 6, 10, 10, d, 16).check()


def test_caller_workspace_of_any_content():
    c = Case(20, [(6000, 1), (70, 1)], 8, 2, 128, 16)
    n = gdn.gdn_paged_attention_kv4_workspace_size(2, 2, 8, 2, 128, 6000)
    want = c.want()
    for fill in (0, 255):
        ws = torch.full((n + 64,), fill, dtype=torch.uint8, device="cuda")
        c.near(c.run(workspace=ws), *want)
        assert (ws[n:] == fill).all()


def test_cache_past_4_gib():
    hk, page, d = 4, 64, 256
    pages = 2 ** 33 // (hk * page * d) + 20
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")                      # noqa: E731
    big = dict(k_cache=u8(pages, hk, page, d // 2), v_cache=u8(pages, hk, page // 16, d, 8), k_scale=u8(pages, hk, d // 32, page),
               v_scale=torch.zeros(pages, hk, page, dtype=torch.bfloat16, device="cuda"))
    c = Case(21, [(100, 1), (150, 20)], 8, hk, d, page)
    at = pages - 1 - np.arange(c.kq.shape[0])
    g = c.gpu()
    for name in big:
        big[name][at.tolist()] = g[name]
    table = np.where(c.table >= 0, at[np.maximum(c.table, 0)], -1)
    g.update(big, block_table=cuda(table, torch.int32))
    o = torch.full(c.q.shape, 77.0, dtype=torch.bfloat16, device="cuda")
    gdn.gdn_paged_attention_kv4(c.q, o=o, max_seq_len=150, scale=c.scale, **g)
    torch.cuda.synchronize()
    c.near(o, *c.want())


@pytest.mark.parametrize("d,page", [(64, 32), (128, 16), (128, 64), (256, 16)])
@pytest.mark.parametrize("lens,longest", [([(5, 1), (2000, 1), (70, 1), (0, 1), (6001, 1), (130, 1)], 2 ** 21),
                                          ([(1 + 37 * i % 700, 1) for i in range(130)], 60000),
                                          ([(300, 2), (65, 0), (0, 0), (900, 1), (40, 1), (3, 0)], 2 ** 21),
                                          ([(300, 90), (2000, 1), (70, 1), (4000, 3)], 2 ** 21)])
def test_a_pool_that_no_cache_holds(d, page, lens, longest):
    """A bound of the lengths and a pool of more than 128 MiB: few rows read it another way."""
    hk = 2
    c = Case(50 + d, lens, 8, hk, d, page)
    pages = 2 ** 27 // (hk * page * d) + 20
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")                      # noqa: E731
    big = dict(k_cache=u8(pages, hk, page, d // 2), v_cache=u8(pages, hk, page // 16, d, 8), k_scale=u8(pages, hk, d // 32, page),
               v_scale=torch.zeros(pages, hk, page, dtype=torch.bfloat16, device="cuda"))
    at = pages - 1 - np.arange(c.kq.shape[0])
    g = c.gpu()
    for name in big:
        big[name][at.tolist()] = g[name]
    table = np.where(c.table >= 0, at[np.maximum(c.table, 0)], -1)
    g.update(big, block_table=cuda(table, torch.int32))
    for window in (0, 100):
        o = torch.full(c.q.shape, 77.0, dtype=torch.bfloat16, device="cuda")
        gdn.gdn_paged_attention_kv4(c.q, o=o, max_seq_len=longest, scale=c.scale, window=window, **g)
        torch.cuda.synchronize()
        c.near(o, *c.want(window=window))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_repeats_are_bit_identical(d):
    c = Case(22, MIXED + [(3000, 1)], 8, 2, d, 16)
    a = c.run()
    for _ in range(3):
        assert torch.equal(a, c.run())


def test_on_a_stream_of_its_own_and_in_a_graph():
    c = Case(23, [(3000, 1), (70, 1), (40, 20)], 8, 2, 128, 16)
    g = c.gpu()
    o = torch.empty_like(c.q)
    n = gdn.gdn_paged_attention_kv4_workspace_size(22, 3, 8, 2, 128, 3000)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    want = c.run()

    def step():
        gdn.gdn_paged_attention_kv4(c.q, o=o, max_seq_len=3000, scale=c.scale, workspace=ws, **g)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    assert torch.equal(o, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        o.zero_()
        g["seq_lens"].copy_(cuda([3000 - 500 * i, 70, 40], torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = o.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, o)


@pytest.mark.parametrize("seed", range(40))
def test_random_batches(seed):
    """Sizes, masks, bounds and missing pages in combinations that no other test here names."""
    r = np.random.default_rng(1000 + seed)
    pick = lambda *x: x[r.integers(len(x))]                                                # noqa: E731
    d, page, hk = pick(64, 128, 256), pick(16, 32, 64), pick(1, 1, 2, 3, 8)
    hq = hk * pick(1, 2, 3, 4, 5, 8, 16)
    lens = []
    for _ in range(pick(1, 2, 3, 5, 17, 40)):
        kind, length = r.random(), int(2 ** r.uniform(0, 11.2))
        new = int(2 ** r.uniform(0, 7.2))
        lens.append((pick(0, -3, 1, 3), pick(0, 1, 2)) if kind < 0.15 else (length, pick(1, 1, 1, 2, 4)) if kind < 0.8 else
                    (new + pick(0, length), new))
    lens.append((int(2 ** r.uniform(0, 11.2)), 1))
    c = Case(seed, lens, hq, hk, d, page, spread=pick(1.0, 3.0))
    if r.random() < 0.3:
        c.table[r.random(c.table.shape) < 0.1] = -1
    for _ in range(2):
        c.check(pick(None, 1, 100, 1000, 2 ** 31 - 1), most=1.0, causal=bool(r.random() < 0.8),
                window=pick(0, 0, 1, 16, 63, 65, 200, 512, 1024, 1500))
