"""GPU checks of gdn_paged_attention_kv8 against the formula in 64 bits.

Bound per element: 2^-8 |o| for the final rounding to bf16, and for the
weights' own rounding to bf16 2^-8 sum_j w_j |v_j|; scores, exponentials and
sums in fp32, and q's split to within 2^-18 of its largest element, are
covered by 2^-10 sum_j w_j |v_j| at the score sizes used here (|x| below 60)."""
import numpy as np
import pytest
import torch

import gated_deltanet_token_amd as gdn
import serving_ref as ref

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def cuda(a, dt):
    return torch.tensor(np.asarray(a), device="cuda").to(dt)


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
        self.kq, self.ks = ref.quantised(r.standard_normal(shape) * np.exp(0.5 * r.standard_normal((pages, hk, 1, 1))))
        vq, self.vs = ref.quantised(r.standard_normal(shape) * np.exp(2 * r.standard_normal((pages, hk, 1, 1))))
        self.vq = vq.transpose(0, 1, 3, 2).copy()
        self.q = cuda((spread * r.standard_normal((T, hq, d))).astype(np.float32), torch.bfloat16)
        self.scale = d ** -0.5
        # what lies past a request's end is anybody's: NaN codes
        for s in range(S):
            L = max(int(self.seq[s]), 0)
            if L % page:
                p = self.table[s, L // page]
                self.kq[p, :, L % page:], self.vq[p, :, :, L % page:] = np.nan, np.nan

    def gpu(self):
        f8 = lambda x: cuda(x.astype(np.float32), torch.float32).to(F8)                 # noqa: E731
        return dict(k_cache=f8(self.kq), v_cache=f8(self.vq), k_scale=cuda(self.ks, torch.float32),
                    v_scale=cuda(self.vs, torch.float32), block_table=cuda(self.table, torch.int32),
                    seq_lens=cuda(self.seq, torch.int32), query_start_loc=cuda(self.qsl, torch.int32))

    def longest(self):
        return max(int(self.seq.max(initial=1)), 1)

    def want(self, **kw):
        return ref.attention(ref.values(self.q), self.kq, self.vq, self.ks, self.vs, self.table, self.seq, self.qsl, self.scale, **kw)

    def run(self, longest=None, q=None, **kw):
        q = self.q if q is None else q
        o = torch.full(q.shape, 77.0, dtype=torch.bfloat16, device="cuda")
        gdn.gdn_paged_attention_kv8(q, o=o, max_seq_len=longest or self.longest(), scale=self.scale, **self.gpu(), **kw)
        torch.cuda.synchronize()
        return o

    def check(self, longest=None, **kw):
        o = self.run(longest, **kw)
        near(o, *self.want(**kw))
        return o


def near(o, want, mag):
    got = ref.values(o)
    owned = ~(mag < 0).all(-1)
    assert (got[~owned] == 77.0).all()
    assert np.array_equal(np.isnan(got[owned]), np.isnan(want[owned]))
    err = np.abs(got - want)[owned]
    bound = (np.abs(want) * 2.0 ** -8 + mag * (2.0 ** -8 + 2.0 ** -10) + 1e-30)[owned]
    fine = ~np.isnan(want[owned])
    assert (err[fine] <= bound[fine]).all(), "%.3g of the bound" % (err[fine] / bound[fine]).max()


DECODE = [(1, 1), (15, 1), (16, 1), (17, 1), (63, 1), (64, 1), (65, 1), (200, 1), (1030, 1)]
MIXED = [(70, 1), (33, 33), (5, 1), (150, 40), (0, 0), (40, 0), (300, 17), (64, 64), (129, 2)]
HEADS = [(1, 1), (4, 4), (8, 2), (5, 1), (16, 2), (16, 1), (24, 1), (40, 2)]


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
def test_long_decode_in_parts(d):
    """Few rows over long contexts: the work is split along the keys and joined."""
    c = Case(4, [(9000, 1), (4097, 1), (3, 1)], 4, 1, d, 32, spread=4.0)
    c.check()
    c.check(window=5000)


@pytest.mark.parametrize("n", [1, 3])
def test_max_seq_len_is_only_a_hint(n):
    c = Case(5, [(5000, n), (100, n)], 8, 2, 128, 16)
    want = c.want()
    for longest in (1, 100, 4999, 5000, 2 ** 31 - 1):
        near(c.run(longest), *want)


def test_rows_without_keys_are_zero():
    """More new tokens than keys, empty requests with tokens, lengths below zero."""
    c = Case(6, [(3, 10), (0, 4), (-7, 2), (20, 40)], 4, 2, 128, 16)
    o = c.check()
    assert (o[:7] == 0).all() and (o[10:16] == 0).all() and (o[16:36] == 0).all()
    c.check(causal=False)


def test_missing_pages_are_not_seen():
    c = Case(7, [(100, 1), (90, 30), (40, 1), (400, 2)], 4, 2, 64, 16)
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
def test_bad_values_reach_only_the_rows_that_see_them(d, hq, hk):
    """NaN codes of a key or value: rows before it keep their results, rows after it are NaN."""
    page = 16
    c = Case(9, [(90, 90), (50, 1), (130, 70)], hq, hk, d, page)
    c.vq[c.table[0, 3], 0, 5, 7] = np.nan          # request 0, key 55: one element
    c.kq[c.table[2, 6], 0, 4, 1] = np.nan          # request 2, key 100
    want, mag = c.want()
    assert np.isnan(want).any() and not np.isnan(want).all()
    got = ref.values(c.run())
    G = hq // hk
    assert np.isnan(got[55:90, :G, 5]).all() and not np.isnan(got[:55]).any() and not np.isnan(got[90]).any()
    near(c.run(), want, mag)
    # NaN scales and codes on pages that nobody's mask reaches
    c = Case(10, [(64, 1), (64, 64)], hq, hk, d, page)
    c.ks[c.table[0, 0]], c.vs[c.table[0, 0]] = np.nan, np.inf
    c.kq[c.table[0, 0]], c.vq[c.table[0, 0]] = np.nan, np.nan
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
    near(got, want, mag)


def test_queries_of_uneven_size():
    """A few elements a thousand times the others, and tiny ones: q's two parts keep them."""
    c = Case(12, [(300, 20), (80, 1)], 4, 2, 128, 16, spread=0.02)
    c.q[:, :, 5] *= 500
    c.check()
    c.q.mul_(2.0 ** -120)
    c.scale *= 2.0 ** 120
    c.check()
    c.q.zero_()
    c.check()


def test_scales_need_not_be_powers_of_two():
    c = Case(13, MIXED, 8, 2, 64, 32)
    c.ks *= c.r.uniform(0.5, 2, c.ks.shape)
    c.vs *= c.r.uniform(0.5, 2, c.vs.shape)
    c.ks, c.vs = c.ks.astype(np.float32), c.vs.astype(np.float32)
    c.check()


@pytest.mark.parametrize("d", [64, 256])
def test_value_scales_far_apart(d):
    c = Case(14, [(200, 1), (200, 60)], 4, 1, d, 16)
    c.vs[::2] *= 2.0 ** 40
    c.vs[1::2] *= 2.0 ** -60
    c.check()


def test_large_scores():
    """One key dominates; fully negative rows; the running maximum moves by hundreds."""
    c = Case(15, [(500, 3), (100, 100)], 4, 2, 64, 16, spread=1.0)
    c.scale = 0.9
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
    gdn.gdn_paged_attention_kv8(qv, o=ov[:, 1:9], max_seq_len=300, scale=c.scale, **g)
    torch.cuda.synchronize()
    near(ov[:T, 1:9], *c.want())
    assert (ov[T:] == 77).all() and (ov[:, 0] == 77).all() and (ov[:, 9] == 77).all()


def test_malformed_query_start_loc_stays_inside():
    c = Case(17, [(50, 10), (60, 10), (70, 10)], 4, 2, 64, 16)
    c.qsl = np.array([0, 25, 12, 900], np.int32)         # a decreasing and a far bound
    c.run()


def test_more_requests_than_a_wave():
    r = np.random.default_rng(18)
    lens = [(int(r.integers(1, 60)), int(r.integers(0, 3))) for _ in range(150)]
    lens = [(max(L, n), n) for L, n in lens]
    Case(18, lens, 4, 2, 64, 16).check()
    Case(19, [(int(r.integers(1, 60)), 1) for _ in range(300)], 4, 2, 64, 16).check()


def test_caller_workspace_of_any_content():
    c = Case(20, [(6000, 1), (70, 1)], 8, 2, 128, 16)
    n = gdn.gdn_paged_attention_kv8_workspace_size(2, 2, 8, 2, 128, 6000)
    want = c.want()
    for fill in (0, 255):
        ws = torch.full((n + 64,), fill, dtype=torch.uint8, device="cuda")
        near(c.run(workspace=ws), *want)
        assert (ws[n:] == fill).all()


def test_cache_past_4_gib():
    hk, page, d = 4, 64, 256
    pages = 2 ** 32 // (hk * page * d) + 20
    k = torch.zeros(pages, hk, page, d, dtype=torch.uint8, device="cuda").view(F8)
    v = torch.zeros(pages, hk, d, page, dtype=torch.uint8, device="cuda").view(F8)
    ks, vs = torch.zeros(pages, hk, device="cuda"), torch.zeros(pages, hk, device="cuda")
    c = Case(21, [(100, 1), (150, 20)], 8, hk, d, page)
    at = pages - 1 - np.arange(c.kq.shape[0])
    g = c.gpu()
    k.view(torch.uint8)[at.tolist()], v.view(torch.uint8)[at.tolist()] = g["k_cache"].view(torch.uint8), g["v_cache"].view(torch.uint8)
    ks[at.tolist()], vs[at.tolist()] = g["k_scale"], g["v_scale"]
    table = np.where(c.table >= 0, at[np.maximum(c.table, 0)], -1)
    g.update(k_cache=k, v_cache=v, k_scale=ks, v_scale=vs, block_table=cuda(table, torch.int32))
    o = torch.full(c.q.shape, 77.0, dtype=torch.bfloat16, device="cuda")
    gdn.gdn_paged_attention_kv8(c.q, o=o, max_seq_len=150, scale=c.scale, **g)
    torch.cuda.synchronize()
    near(o, *c.want())


def test_repeats_are_bit_identical():
    c = Case(22, MIXED + [(3000, 1)], 8, 2, 128, 16)
    a = c.run()
    for _ in range(3):
        assert torch.equal(a, c.run())


def test_on_a_stream_of_its_own_and_in_a_graph():
    c = Case(23, [(3000, 1), (70, 1), (40, 20)], 8, 2, 128, 16)
    g = c.gpu()
    o = torch.empty_like(c.q)
    n = gdn.gdn_paged_attention_kv8_workspace_size(22, 3, 8, 2, 128, 3000)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    want = c.run()

    def step():
        gdn.gdn_paged_attention_kv8(c.q, o=o, max_seq_len=3000, scale=c.scale, workspace=ws, **g)

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


@pytest.mark.parametrize("d", [64, 128, 256])
def test_value_scales_over_their_whole_range(d):
    """Every page's scale another one from 2^-100 to 2^100, not powers of two, some zero or
    negative: none passes fp32's end in a weight, none's rounding reaches another row."""
    c = Case(19, [(300, 70), (90, 90), (500, 1), (64, 40)], 8, 2, d, 16, spread=2.0)
    c.vs = (2.0 ** c.r.integers(-100, 101, c.vs.shape) * c.r.uniform(1, 2, c.vs.shape)).astype(np.float32)
    c.vs[::7] = 0
    c.vs[1::5] *= -1
    c.check()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("step", [1.0, 7.5, 8.5, 200.0])
def test_scores_that_rise_or_fall_with_the_key(d, step):
    """The running maximum moves by `step` powers of two per 16 keys, up in one kv head and
    down in the other: sums follow it at once, late, or not at all."""
    c = Case(20, [(200, 100), (330, 1), (150, 33)], 4, 2, d, 16, spread=0.0)
    c.q[...] = 0
    c.q[:, :, 0] = 1.0
    c.kq[...] = 0
    c.kq[:, :, :, 0] = 256.0
    c.scale = 2.0 ** -8 * np.log(2.0)
    for s in range(len(c.seq)):
        for i in range(-(-int(c.seq[s]) // 16)):
            c.ks[c.table[s, i]] = [step * (i + 1), step * (40 - i)]
    c.check()
