"""GPU checks of gdn_build_step_tables against a request-by-request reference:
every output exactly, at sizes and shortages where it can go wrong."""
import numpy as np
import pytest
import torch

import gated_deltanet_token_amd as gdn
import serving_ref as ref

pytestmark = pytest.mark.gpu


def t32(a):
    return torch.tensor(np.asarray(a, np.int32), dtype=torch.int32, device="cuda")


def call(ctx, new, free, num_free, table, page, T, n_chunks, stride=None, stream=None):
    S, cols = table.shape
    wide = torch.full((S, stride or cols), -7, dtype=torch.int32, device="cuda")
    bt = wide[:, :cols]
    bt.copy_(t32(table))
    out = dict(query_start_loc=t32(np.full(S + 1, -9)), seq_lens=t32(np.full(S, -9)), positions=t32(np.full(T, -9)),
               slot_mapping=torch.full((T,), -9, dtype=torch.int64, device="cuda"), counts=t32(np.full(4, -9)))
    chunks = t32(np.full((n_chunks, 2), -9)) if n_chunks else None
    gdn.gdn_build_step_tables(t32(ctx), t32(new), t32(free), t32([num_free]), bt, page, out["query_start_loc"], out["seq_lens"],
                              out["positions"], out["slot_mapping"], out["counts"], chunks=chunks, stream=stream)
    torch.cuda.synchronize()
    assert (wide[:, cols:] == -7).all()
    got = [out["query_start_loc"], out["seq_lens"], out["positions"], out["slot_mapping"], bt, chunks, out["counts"]]
    return [np.zeros((0, 2), np.int32) if x is None else x.cpu().numpy() for x in got]


def check(ctx, new, free, num_free, table, page, T, n_chunks, **kw):
    got = call(ctx, new, free, num_free, table, page, T, n_chunks, **kw)
    want = ref.tables(ctx, new, np.asarray(free), num_free, np.asarray(table), page, T, n_chunks)
    for name, g, w in zip(("query_start_loc", "seq_lens", "positions", "slots", "table", "chunks", "counts"), got, want):
        assert g.shape == w.shape and np.array_equal(g, w), name
    return got


def batch(r, S, page, longest, most_new, idle=0.2):
    ctx = r.integers(0, longest + 1, S) * (r.random(S) < 0.9)
    new = np.where(r.random(S) < 0.6, 1, r.integers(0, most_new + 1, S)) * (r.random(S) >= idle)
    cols = int(-(-(ctx + new).max() // page)) if S else 1
    cols = max(cols, 1)
    held = -(-ctx // page)
    need = int((-(-(ctx + new) // page) - held).sum())
    ids = r.permutation(int(held.sum()) + need + 5)
    table = np.full((S, cols), -1, np.int32)
    at = 0
    for s in range(S):
        table[s, :held[s]] = ids[at:at + held[s]]
        at += held[s]
    return ctx, new, ids[at:], table, need


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    r = np.random.default_rng(seed)
    S = int(r.choice([1, 2, 3, 31, 64, 65, 300, 1023, 1025]))
    page = int(r.choice([1, 8, 16, 32, 64, 1024]))
    ctx, new, free, table, need = batch(r, S, page, int(r.choice([0, 5, 100, 3000])), int(r.choice([1, 7, 8, 9, 200])))
    T, n = int(new.sum()), int((-(-new // 8)).sum())
    got = check(ctx, new, free, len(free), table, page, T, n)
    assert got[6].tolist() == [T, n, need, 0]
    if n:
        assert np.array_equal(got[5], gdn.gdn_build_conv_chunks(got[0]))


@pytest.mark.parametrize("spare", [-3, -1, 0, 1, 2, 500])
def test_outputs_shorter_and_longer_than_the_step(spare):
    r = np.random.default_rng(5)
    ctx, new, free, table, _ = batch(r, 40, 16, 300, 90)
    T, n = int(new.sum()), int((-(-new // 8)).sum())
    check(ctx, new, free, len(free), table, 16, max(T + spare, 0), max(n + spare, 0))


@pytest.mark.parametrize("left", [0, 1, 7, -4])
def test_free_list_runs_out(left):
    r = np.random.default_rng(6)
    ctx, new, free, table, need = batch(r, 50, 16, 200, 60, idle=0.0)
    got = check(ctx, new, free, left, table, 16, int(new.sum()), 400)
    assert need > 7 and got[6][2] == max(left, 0) and got[6][3] == need - max(left, 0)


def test_num_free_past_the_list_is_clamped():
    r = np.random.default_rng(7)
    ctx, new, free, table, _ = batch(r, 9, 16, 100, 60)
    a = call(ctx, new, free, len(free) + 1000, table, 16, int(new.sum()), 100)
    b = call(ctx, new, free, len(free), table, 16, int(new.sum()), 100)
    assert all(np.array_equal(x, y) for x, y in zip(a, b))


def test_full_rows():
    """Requests whose pages pass the row's end: their later tokens have no slot."""
    table = np.full((4, 3), -1, np.int32)
    table[0, :3], table[1, :2] = [5, 6, 7], [8, 9]
    got = check([48, 30, 0, 100], [5, 40, 200, 3], np.arange(20, 40), 20, table, 16, 248, 40, stride=8)
    assert got[6][3] == 1 + 2 + 10 and (got[3][:5] == -1).all()


def test_negative_lengths_count_as_zero():
    table = np.full((3, 4), -1, np.int32)
    check([-5, 3, 0], [4, -2, 17], np.arange(9), 9, table, 16, 30, 9)


def test_nothing():
    got = check([], [], [4, 5], 2, np.zeros((0, 3), np.int32), 16, 3, 2)
    assert got[0].tolist() == [0] and got[6].tolist() == [0, 0, 0, 0]
    check([3, 0], [0, 0], [], 0, np.full((2, 1), 9, np.int32), 16, 0, 0)


def test_most_requests_and_many_tokens():
    r = np.random.default_rng(8)
    ctx, new, free, table, need = batch(r, gdn.STEP_MAX_SEQS, 16, 900, 30, idle=0.1)
    new[17] = 30000
    cols = -(-int((ctx + new).max()) // 16)
    wide = np.full((len(ctx), cols), -1, np.int32)
    wide[:, :table.shape[1]] = table
    free = np.arange(10 ** 6, 10 ** 6 + 60000)
    check(ctx, new, free, len(free), wide, 16, int(new.sum()) + 3, int((-(-new // 8)).sum()) + 3)


def test_long_contexts_and_slots_past_32_bits():
    ctx, new = [2 ** 31 - 100, 5], [50, 3]
    table = np.full((2, 2 ** 21), -1, np.int32)
    table[0, :] = 2 ** 31 - 1
    table[1, 0] = 2 ** 31 - 5
    got = check(ctx, new, [], 0, table, 1024, 53, 9)
    assert got[3].min() > 2 ** 40


def test_sums_saturate():
    got = call([2 ** 31 - 1, 2 ** 31 - 1], [2 ** 31 - 1, 2 ** 31 - 1], [3], 1, np.zeros((2, 1), np.int32), 1024, 5, 5)
    top = 2 ** 31 - 1
    assert got[0].tolist() == [0, top, top] and got[1].tolist() == [top, top] and got[6][0] == top
    assert (got[3] == -1).all() and got[2].tolist() == [top] * 5


def test_on_a_stream_of_its_own_and_in_a_graph():
    r = np.random.default_rng(9)
    ctx, new, free, table, _ = batch(r, 64, 16, 300, 20)
    T, n = int(new.sum()), int((-(-new // 8)).sum())
    a = call(ctx, new, free, len(free), table, 16, T, n)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    i = [t32(ctx), t32(new), t32(free), t32([len(free)]), t32(table)]
    o = [t32(np.zeros(65)), t32(np.zeros(64)), t32(np.zeros(T)), torch.zeros(T, dtype=torch.int64, device="cuda"), t32(np.zeros(4))]
    ch = t32(np.zeros((n, 2)))
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        gdn.gdn_build_step_tables(*i, 16, *o, chunks=ch)
    s.synchronize()
    assert np.array_equal(o[3].cpu().numpy(), a[3])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gdn.gdn_build_step_tables(*i, 16, *o, chunks=ch)
    for step in range(3):                       # lengths change between replays, on the device
        i[0].copy_(t32(ctx + 16 * step))        # whole pages: the rows' entries below stay
        i[4].copy_(t32(np.concatenate([np.full((64, step), 3), table[:, :table.shape[1] - step]], 1)))
        before = i[4].cpu().numpy()
        g.replay()
        torch.cuda.synchronize()
        want = ref.tables(ctx + 16 * step, new, free, len(free), before, 16, T, n)
        got = [o[0], o[1], o[2], o[3], i[4], ch, o[4]]
        assert all(np.array_equal(x.cpu().numpy(), w) for x, w in zip(got, want))
