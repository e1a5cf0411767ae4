"""GPU checks of examples/hybrid_step.py, which runs the step tables, the norms,
the Gated DeltaNet calls, the cache append and the attention together."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_step.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("hybrid_step", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def prompts(example, lens, seed):
    stack = example.HybridStack(len(lens), max_len=128, seed=seed)
    x = torch.randn(sum(lens), example.HIDDEN, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")
    h, t = stack.step(x.to(torch.bfloat16), torch.tensor(lens, dtype=torch.int32, device="cuda"), max(lens))
    return stack, h, t


def test_tables_of_the_steps(example):
    lens = [17, 1, 40, 16]
    stack, h, t = prompts(example, lens, 3)
    assert h.isfinite().all() and stack.context_lens.tolist() == lens
    held = [-(-n // example.PAGE) for n in lens]
    total = stack.free_pages.shape[0]
    assert t["counts"].tolist() == [sum(lens), sum(-(-n // 8) for n in lens), sum(held), 0]
    one = torch.ones(len(lens), dtype=torch.int32, device="cuda")
    x = h[t["query_start_loc"][1:].long() - 1].clone()
    for _ in range(20):
        x, t = stack.step(x, one, 128, decode=True)
        assert x.isfinite().all()
    lens = [n + 20 for n in lens]
    held = [-(-n // example.PAGE) for n in lens]
    assert stack.context_lens.tolist() == lens and int(stack.num_free) == total - sum(held)
    taken = [p for row, n in zip(stack.block_table.tolist(), held) for p in row[:n]]
    assert sorted(taken) == sorted(stack.free_pages.tolist()[int(stack.num_free):])


def test_a_decode_step_replayed_as_a_graph_is_the_same(example):
    lens, steps = [15, 33, 1], 6
    stack, h, t = prompts(example, lens, 4)
    one = torch.ones(len(lens), dtype=torch.int32, device="cuda")
    first = h[t["query_start_loc"][1:].long() - 1].clone()
    want, x = [], first
    for _ in range(steps):
        x, _ = stack.step(x, one, 128, decode=True)
        want.append(x.clone())

    stack, h2, _ = prompts(example, lens, 4)
    assert torch.equal(h, h2)
    x = first.clone()
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
        torch.ones(1000, device="cuda").sum()          # eager work between the replays
