"""GPU checks of gdn_paged_read_kv4: keys are exact in bf16, values codes times
scales rounded once to bf16 (both equal to what numpy and torch make of them)."""
import numpy as np
import pytest
import torch

import gated_deltanet_token_amd as gdn
import kv4_ref as kv4

pytestmark = pytest.mark.gpu


class Cache:
    """A cache of random codes and scales of the usual sizes, and its values."""

    def __init__(self, seed, pages, hk, page, d):
        r = self.r = np.random.default_rng(seed)
        self.kq, self.vq = (r.integers(0, 16, (pages, hk, page, d), dtype=np.uint8) for _ in range(2))
        self.ks = r.integers(110, 140, (pages, hk, page, d // 32)).astype(np.uint8)
        self.vs = kv4.bf16(np.exp(r.standard_normal((pages, hk, page))))

    def gpu(self):
        t = lambda x: torch.tensor(x, device="cuda")                                       # noqa: E731
        return dict(k_cache=t(kv4.pack_k(self.kq)), v_cache=t(kv4.pack_v(self.vq)), k_scale=t(kv4.pack_k_scale(self.ks)),
                    v_scale=t(self.vs.astype(np.float32)).to(torch.bfloat16))

    def rows(self):
        """k and v [pages * page][hk][D] as bf16"""
        n = self.kq.shape[0] * self.kq.shape[2]
        f = lambda x: torch.tensor(x.swapaxes(1, 2).reshape(n, *x.shape[1:2], -1)).to(torch.bfloat16)   # noqa: E731
        return f(kv4.key_values(self.kq, self.ks)), f(kv4.value_values(self.vq, self.vs))


def i32(a):
    return torch.tensor(np.asarray(a, np.int32), device="cuda")


def check(c, table, starts, loc, rows=None, stride_heads=None):
    pages, hk, page, d = c.kq.shape
    R = int(loc[-1]) if rows is None else rows
    wide = stride_heads or hk
    k, v = (torch.full((R, wide, d), 77.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bt = i32(table)
    gdn.gdn_paged_read_kv4(**c.gpu(), block_table=bt, key_starts=None if starts is None else i32(starts), out_start_loc=i32(loc),
                           k_out=k[:, :hk], v_out=v[:, :hk])
    torch.cuda.synchronize()
    want = [torch.full((R, wide, d), 77.0, dtype=torch.bfloat16) for _ in range(2)]
    of = c.rows()
    for s in range(len(loc) - 1):
        a, b = min(max(int(loc[s]), 0), R), min(max(int(loc[s + 1]), 0), R)
        for i in range(a, b):
            j = (0 if starts is None else max(int(starts[s]), 0)) + i - a
            p = table[s][j // page] if j // page < len(table[s]) else -1
            if 0 <= p < pages:
                for w, x in zip(want, of):
                    w[i, :hk] = x[p * page + j % page]
    for got, w in zip((k, v), want):
        got = got.cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(w))
        assert torch.equal(got.nan_to_num(5.0), w.nan_to_num(5.0))
    return k, v


def table_of(c, lens):
    pages, page = c.kq.shape[0], c.kq.shape[2]
    ids = list(c.r.permutation(pages))
    need = [-(-n // page) for n in lens]
    table = np.full((len(lens), max(need) + 1), -1, np.int64)
    for s, n in enumerate(need):
        table[s, :n] = [ids.pop() for _ in range(n)]
    return table


@pytest.mark.parametrize("d,page", [(64, 16), (64, 64), (128, 32), (128, 16), (256, 16), (256, 64)])
@pytest.mark.parametrize("hk", [1, 2, 3, 4, 8, 9])
def test_ranges(d, page, hk):
    c = Cache(d + page + hk, 60, hk, page, d)
    starts = [0, 5, 16, 31, 17, 0, 15, 40, 3]
    n = [1, 3, 16, 33, 0, 100, 2, 47, 13]
    table = table_of(c, [a + b for a, b in zip(starts, n)])
    check(c, table, starts, np.concatenate([[0], np.cumsum(n)]))
    check(c, table, None, np.concatenate([[0], np.cumsum([1, 8, 30, 60, 0, 100, 5, 80, 16])]))


def test_many_requests_and_empty_ones():
    c = Cache(1, 400, 2, 16, 64)
    n = c.r.integers(0, 20, 300)
    starts = c.r.integers(0, 5, 300)
    n[100:170] = 0
    check(c, table_of(c, (starts + n).tolist()), starts, np.concatenate([[0], np.cumsum(n)]))


def test_only_keys_or_only_values():
    c = Cache(2, 10, 4, 32, 128)
    table, loc = table_of(c, [70, 40]), [0, 70, 110]
    k, v = check(c, table, None, loc)
    for which in (0, 1):
        out = torch.full_like(k, 5.0)
        outs = dict(k_out=out, v_out=None) if which == 0 else dict(k_out=None, v_out=out)
        gdn.gdn_paged_read_kv4(**c.gpu(), block_table=i32(table), key_starts=None, out_start_loc=i32(loc), **outs)
        assert torch.equal(out, (k, v)[which])


def test_strided_rows_and_a_strided_table():
    c = Cache(3, 10, 3, 16, 64)
    table = table_of(c, [50, 30])
    check(c, table, [3, 0], [0, 40, 70], rows=90, stride_heads=7)
    bt = torch.full((2, 40), -1, dtype=torch.int32, device="cuda")
    bt[:, :table.shape[1]] = i32(table)
    k, v = (torch.zeros(70, 3, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gdn.gdn_paged_read_kv4(**c.gpu(), block_table=bt[:, :table.shape[1]], key_starts=i32([3, 0]), out_start_loc=i32([0, 40, 70]),
                           k_out=k, v_out=v)
    a, b = check(c, table, [3, 0], [0, 40, 70])
    assert torch.equal(k, a) and torch.equal(v, b)


def test_missing_pages_and_the_rows_end_leave_rows_alone():
    c = Cache(4, 12, 2, 16, 64)
    table = table_of(c, [80, 60, 30])
    table[0, 1], table[1, 0], table[1, 2], table[2, 1] = -1, 12, 2 ** 31 - 1, -2 ** 31
    check(c, table, [0, 7, -9], [0, 80, 140, 300])             # the last one reaches past its row of pages
    check(c, table, [2 ** 31 - 1, 70, 2 ** 31 - 20], [0, 30, 60, 90])


def test_malformed_out_start_loc_stays_inside():
    c = Cache(4, 12, 2, 16, 64)
    out = torch.full((110, 2, 64), 77.0, dtype=torch.bfloat16, device="cuda")
    gdn.gdn_paged_read_kv4(**c.gpu(), block_table=i32(table_of(c, [80, 60, 30])), key_starts=None,
                           out_start_loc=i32([0, 50, 20, 900]), k_out=out[:100], v_out=None)      # a decreasing and a far bound
    assert (out[100:] == 77.0).all()


def test_scales_over_their_whole_range():
    c = Cache(5, 16, 2, 16, 64)
    c.ks[...] = np.arange(c.ks.size).reshape(c.ks.shape) % 254     # down to 2^-127: values down to bf16's subnormal ones
    c.ks[3, 0, 4, 1] = 255
    c.vs = kv4.bf16(np.exp2(c.r.uniform(-118, 124, c.vs.shape)))
    c.vs[5, 1, 7] = np.nan
    table = np.arange(16)[None]
    check(c, table, None, [0, 256])


def test_cache_past_4_gib():
    hk, page, d = 4, 64, 256
    pages = 2 ** 33 // (hk * page * d) + 20
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")                      # noqa: E731
    cache = dict(k_cache=u8(pages, hk, page, d // 2), v_cache=u8(pages, hk, page // 16, d, 8), k_scale=u8(pages, hk, d // 32, page),
                 v_scale=torch.zeros(pages, hk, page, dtype=torch.bfloat16, device="cuda"))
    c = Cache(6, 3, hk, page, d)
    for name, t in c.gpu().items():
        cache[name][-3:] = t
    table, loc = [[0, 2, 1]], [0, 150]
    want = check(c, np.array(table), [20], loc)
    k, v = torch.empty_like(want[0]), torch.empty_like(want[1])
    gdn.gdn_paged_read_kv4(**cache, block_table=i32(np.array(table) + pages - 3), key_starts=i32([20]), out_start_loc=i32(loc), k_out=k,
                           v_out=v)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


def test_on_a_stream_of_its_own_and_in_a_graph():
    c = Cache(7, 20, 2, 32, 128)
    table, loc = i32(table_of(c, [90, 200])), i32([0, 85, 280])
    starts, g = i32([5, 3]), c.gpu()
    k, v = (torch.zeros(280, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    a, b = torch.zeros_like(k), torch.zeros_like(v)
    gdn.gdn_paged_read_kv4(**g, block_table=table, key_starts=starts, out_start_loc=loc, k_out=a, v_out=b)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    gdn.gdn_paged_read_kv4(**g, block_table=table, key_starts=starts, out_start_loc=loc, k_out=k, v_out=v, stream=side)
    side.synchronize()
    assert torch.equal(k, a) and torch.equal(v, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_paged_read_kv4(**g, block_table=table, key_starts=starts, out_start_loc=loc, k_out=k, v_out=v)
    for i in range(3):
        starts.copy_(i32([i, 2 * i]))
        k.zero_(), v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        gdn.gdn_paged_read_kv4(**g, block_table=table, key_starts=starts, out_start_loc=loc, k_out=a, v_out=b)
        torch.cuda.synchronize()
        assert torch.equal(k, a) and torch.equal(v, b)
