"""GPU checks of the 4-bit paged cache's calls one behind the other, as an engine
makes them: step tables, append, attention and read back, in a batch that changes
from step to step, in graphs that share a workspace, and in examples/hybrid_step.py.

The attention is compared with the formula in 64 bits over what the cache then holds,
with the bound of test_gpu_kv4_attention.py; what is read back with the cache's
codes and scales, exactly."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import gated_deltanet_token_amd as gdn
import kv4_ref as kv4
import serving_ref as ref
from test_gpu_kv4_attention import Case
from test_gpu_serving_attention import cuda

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_step.py")
BF16 = torch.bfloat16


class Engine(Case):
    """S requests, their lengths and pages on the GPU, and one layer's cache."""

    def __init__(self, S, max_len, hq, hk, d, page, seed=0):
        self.r, self.page, self.shape = np.random.default_rng(seed), page, (hq, hk, d)
        columns = -(-max_len // page)
        pages = S * columns
        i32 = dict(dtype=torch.int32, device="cuda")
        self.context, self.bt = torch.zeros(S, **i32), torch.full((S, columns), -1, **i32)
        self.free, self.num_free = cuda(self.r.permutation(pages), torch.int32), torch.full((1,), pages, **i32)
        u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")                  # noqa: E731
        self.cache = dict(k_cache=u8(pages, hk, page, d // 2), v_cache=u8(pages, hk, page // 16, d, 8),
                          k_scale=u8(pages, hk, d // 32, page), v_scale=torch.zeros(pages, hk, page, dtype=BF16, device="cuda"))
        self.frequencies = torch.tensor(10000.0 ** -(np.arange(16) / 16), device="cuda")
        self.scale, self.max_len = d ** -0.5, max_len

    def inputs(self, T):
        hq, hk, d = self.shape
        return cuda(self.r.standard_normal((T, hq + 2 * hk, d)).astype(np.float32), BF16)

    def step(self, x, lens, q, o, t, ws=None, longest=None):
        """The new tokens' q | k | v in x, lens[s] of request s; q: rotated; o: the result."""
        hq, hk, _ = self.shape
        gdn.gdn_build_step_tables(self.context, lens, self.free, self.num_free, self.bt, self.page, t["loc"], t["seq"],
                                  t["pos"], t["slot"], t["counts"], None)
        gdn.gdn_rope_append_kv4(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], t["pos"], t["slot"], self.frequencies, q,
                                **self.cache)
        gdn.gdn_paged_attention_kv4(q, **self.cache, block_table=self.bt, seq_lens=t["seq"], query_start_loc=t["loc"], o=o,
                                    max_seq_len=longest or self.max_len, scale=self.scale, workspace=ws)
        self.context.copy_(t["seq"])
        self.num_free.sub_(t["counts"][2:3])

    def tables(self, T):
        S = self.context.shape[0]
        i32 = dict(dtype=torch.int32, device="cuda")
        return dict(loc=torch.empty(S + 1, **i32), seq=torch.empty(S, **i32), pos=torch.empty(T, **i32),
                    slot=torch.empty(T, dtype=torch.int64, device="cuda"), counts=torch.empty(4, **i32))

    def run(self, lens):
        T = int(sum(lens))
        x, t = self.inputs(T), self.tables(T)
        q = torch.empty(T, self.shape[0], self.shape[2], dtype=BF16, device="cuda")
        o = torch.full_like(q, 77.0)
        self.step(x, cuda(lens, torch.int32), q, o, t)
        torch.cuda.synchronize()
        self.check_step(q, o, t)

    def check_step(self, q, o, t):
        hq, hk, d = self.shape
        c = {n: x.cpu() for n, x in self.cache.items()}
        self.kq, self.vq = kv4.unpack_k(c["k_cache"].numpy()), kv4.unpack_v(c["v_cache"].numpy())
        self.ks, self.vs = c["k_scale"].numpy().swapaxes(2, 3), c["v_scale"].double().numpy()
        self.q, self.table = q, self.bt.cpu().numpy()
        self.seq, self.qsl = t["seq"].cpu().numpy(), t["loc"].cpu().numpy()
        self.near(o, *self.want())
        # every request's keys and values, read back
        loc = np.concatenate([[0], np.cumsum(self.seq)])
        k, v = (torch.full((int(loc[-1]), hk, d), 77.0, dtype=BF16, device="cuda") for _ in range(2))
        gdn.gdn_paged_read_kv4(**self.cache, block_table=self.bt, key_starts=None, out_start_loc=cuda(loc, torch.int32),
                               k_out=k, v_out=v)
        kw, vw = kv4.key_values(self.kq, self.ks), kv4.value_values(self.vq, self.vs)
        for s, n in enumerate(self.seq):
            at = self.table[s, np.arange(n) // self.page], slice(None), np.arange(n) % self.page
            for got, w in ((k, kw), (v, vw)):
                assert torch.equal(got[loc[s]:loc[s + 1]].cpu(), torch.tensor(w[at]).to(BF16))


@pytest.mark.parametrize("hq,hk,d,page", [(4, 2, 64, 16), (8, 2, 128, 32), (4, 4, 256, 16), (6, 1, 256, 64)])
def test_steps_of_an_engine(hq, hk, d, page):
    """Prompts, chunks that continue them, decode rows beside chunks, decode rows, and none."""
    e = Engine(5, 700, hq, hk, d, page)
    for lens in ([37, 0, 200, 1, 64], [1, 300, 41, 1, 0], [1, 1, 1, 30, 1], [1, 1, 1, 1, 1], [1, 0, 0, 1, 0], [90, 1, 1, 2, 300]):
        e.run(lens)
    assert e.context.tolist() == [131, 303, 244, 36, 366]


def test_decode_steps_in_a_graph():
    """The lengths grow on the GPU: each replay is the next step, with the same results as one by one."""
    def engine():
        e = Engine(3, 3000, 8, 2, 128, 16, seed=3)
        e.run([2500, 15, 33])
        return e

    one = torch.ones(3, dtype=torch.int32, device="cuda")
    n = gdn.gdn_paged_attention_kv4_workspace_size(3, 3, 8, 2, 128, 3000)
    e = engine()
    xs, got = [e.inputs(3) for _ in range(7)], []
    x, t, q, ws = torch.empty_like(xs[0]), e.tables(3), torch.empty(3, 8, 128, dtype=BF16, device="cuda"), None
    o = torch.empty_like(q)
    assert n > 0
    for y in xs:
        x.copy_(y)
        e.step(x, one, q, o, t)
        torch.cuda.synchronize()
        e.check_step(q, o, t)
        got.append(o.clone())
    e = engine()
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    x.copy_(xs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        e.step(x, one, q, o, t, ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, got[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        e.step(x, one, q, o, t, ws)
    for y, w in zip(xs[1:], got[1:]):
        x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, w)
        torch.ones(1000, device="cuda").sum()              # eager work between the replays


def test_two_graphs_share_a_workspace():
    """On one stream, in any order: a call leaves nothing in the workspace that another needs."""
    a, b = Case(41, [(6000, 1), (70, 1)], 8, 2, 128, 16), Case(42, [(2500, 1), (900, 40), (4000, 2)], 4, 2, 256, 16)
    n = max(gdn.gdn_paged_attention_kv4_workspace_size(2, 2, 8, 2, 128, 6000),
            gdn.gdn_paged_attention_kv4_workspace_size(43, 3, 4, 2, 256, 4000))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    made = []
    for c in (a, b):
        want, g, o = c.run(), c.gpu(), torch.empty_like(c.q)
        c.near(want, *c.want())
        call = lambda c=c, g=g, o=o: gdn.gdn_paged_attention_kv4(c.q, o=o, max_seq_len=c.longest(), scale=c.scale,   # noqa: E731
                                                                 workspace=ws, **g)
        call()
        torch.cuda.synchronize()
        assert torch.equal(o, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        made.append((graph, o, want, call))
    for i in (0, 1, 1, 0, 1, 0, 0):
        graph, o, want, call = made[i]
        o.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)
        made[1 - i][3]()                                    # the other one's call, eagerly, in between
    for graph, o, _, _ in made:
        o.fill_(5.0)
    made[0][0].replay(), made[1][0].replay(), made[0][0].replay()
    torch.cuda.synchronize()
    for _, o, want, _ in made:
        assert torch.equal(o, want)


def test_two_streams_at_once():
    """Two batches over one cache, each with its stream, tables and workspace."""
    c = Case(43, [(6000, 1), (70, 1), (900, 40)], 8, 2, 128, 16)
    g, want = c.gpu(), c.run()
    n = gdn.gdn_paged_attention_kv4_workspace_size(42, 3, 8, 2, 128, 6000)
    outs = [(torch.cuda.Stream(), torch.empty_like(c.q), torch.empty(n, dtype=torch.uint8, device="cuda")) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o, ws in outs:
            gdn.gdn_paged_attention_kv4(c.q, o=o, max_seq_len=6000, scale=c.scale, workspace=ws, stream=s, **g)
    torch.cuda.synchronize()
    for _, o, _ in outs:
        assert torch.equal(o, want)


def test_a_slot_named_twice_stays_in_its_granule():
    """Which of the two tokens' numbers the slot has is not said, nor what codes the values of its
    granule have; all others are as they were."""
    r = np.random.default_rng(44)
    hk, d, page, pages = 2, 128, 16, 6
    u8 = lambda *s: torch.randint(0, 256, s, dtype=torch.uint8, device="cuda", generator=torch.Generator("cuda").manual_seed(7))  # noqa: E731
    cache = [u8(pages, hk, page, d // 2), u8(pages, hk, page // 16, d, 8), u8(pages, hk, d // 32, page),
             torch.ones(pages, hk, page, dtype=BF16, device="cuda")]
    before = [x.clone() for x in cache]
    slots = cuda([40, 41, 41, 42, 77, 40], torch.int64)
    x = cuda(r.standard_normal((6, 2 * hk + 4, d)).astype(np.float32), BF16)
    q = torch.empty(6, 4, d, dtype=BF16, device="cuda")
    gdn.gdn_rope_append_kv4(x[:, :4], x[:, 4:6], x[:, 6:], cuda(np.arange(6), torch.int32), slots,
                            torch.ones(8, dtype=torch.float64, device="cuda"), q, *cache)
    torch.cuda.synchronize()
    for got, old, i in zip(cache, before, range(4)):
        form = (kv4.unpack_k, kv4.unpack_v, lambda t: t.swapaxes(2, 3), lambda t: t)[i]
        keep = np.ones(pages * page, bool)
        keep[[40, 41, 42, 77]] = False
        if i == 1:
            keep[32:48] = False
        keep = keep.reshape(pages, page)
        a, b = (form(y.view(torch.int16).cpu().numpy() if y.dtype == BF16 else y.cpu().numpy()) for y in (got, old))
        a, b = np.moveaxis(a, 1, 2), np.moveaxis(b, 1, 2)                   # [page][token][head] ..
        assert np.array_equal(a[keep], b[keep])


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("hybrid_step", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_the_hybrid_example(example):
    """Prompts and decode steps of the whole stack; a step replayed as a graph is the same."""
    lens, steps = [15, 33, 1], 5
    one = torch.ones(3, dtype=torch.int32, device="cuda")

    def prompts():
        stack = example.HybridStack(3, max_len=128, seed=4, cache_bits=4)
        x = torch.randn(sum(lens), example.HIDDEN, generator=torch.Generator("cuda").manual_seed(4), device="cuda")
        h, t = stack.step(x.to(BF16), cuda(lens, torch.int32), max(lens))
        return stack, h, h[t["query_start_loc"][1:].long() - 1].clone()

    stack, h, first = prompts()
    assert h.isfinite().all()
    want, x = [], first
    for _ in range(steps):
        x, _ = stack.step(x, one, 128, decode=True)
        want.append(x.clone())
    stack, _, x = prompts()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        h, _ = stack.step(x, one, 128, decode=True)
        x.copy_(h)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(x, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, _ = stack.step(x, one, 128, decode=True)
        x.copy_(h)
    for i in range(1, steps):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, want[i]), "step %d" % i
