"""The scratch that the binding allocates for a call on a given stream comes
from that stream's memory: memory freed a moment ago on the current stream may
still be in use by kernels there, which the given stream does not wait for."""
import contextlib

import pytest
import torch

import gated_deltanet_token_amd as gdn
import synth
from parity import dev


def test_scratch_is_allocated_on_the_calls_stream(monkeypatch):
    """On the CPU, with torch's stream context and allocation recorded."""
    on, got, empty = [None], [], torch.empty

    @contextlib.contextmanager
    def stream(s):
        on.append(s)
        yield
        on.pop()

    def allocate(n, dtype, device):
        got.append((n, dtype, on[-1]))
        return empty(n, dtype=dtype)

    class Stream:
        cuda_stream = 7

    s = Stream()
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "empty", allocate)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda *a: None)
    gdn._workspace(None, 100, torch.device("cuda"), s)
    gdn._workspace(None, 0, torch.device("cuda"), None)
    assert got == [(100, torch.uint8, s), (1, torch.uint8, None)] and on == [None]


def _freed_behind_work(n):
    """A block of n bytes freed on the current stream with a fill of it still to come."""
    junk = torch.empty(n, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(20_000_000)
    for i in range(50):
        junk.fill_(i)
    return junk.data_ptr()


@pytest.mark.gpu
def test_attention_beside_work_on_a_freed_block():
    """Decode rows whose keys are split: partial sums of 256 workgroups."""
    from test_gpu_serving_attention import Case
    c = Case(31, [(9000, 1), (7000, 1), (300, 1)], 16, 2, 128, 16)
    need = gdn.gdn_paged_attention_kv8_workspace_size(3, 3, 16, 2, 128, 9000)
    assert need > 0
    want, g = c.run(), c.gpu()
    o, side = torch.full_like(c.q, 77.0), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        o.fill_(77.0)
        side.wait_stream(torch.cuda.current_stream())
        _freed_behind_work(need)
        gdn.gdn_paged_attention_kv8(c.q, o=o, max_seq_len=9000, scale=c.scale, stream=side, **g)
        torch.cuda.synchronize()
        assert torch.equal(o, want)


@pytest.mark.gpu
def test_chunk_rule_beside_work_on_a_freed_block():
    d = synth.random_gdn(40, 79, [300, 200], 4, 8, 128, 128, num_slots=4, has_init=[1, 0])
    names = ("q", "k", "v", "g", "beta", "state_indices", "qsl", "has_init")
    t = {n: dev(d[n]) for n in names + ("state",)}
    T, HV = t["v"].shape[0], t["v"].shape[1]
    need = gdn.gdn_chunk_workspace_size(2, T, 4, HV)

    def call(stream=None):
        o, st = torch.zeros_like(t["v"]), t["state"].clone()
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
            _freed_behind_work(need)
        gdn.gdn_chunk_gated_delta_rule(*(t[n] for n in names[:5]), st, t["state_indices"], o, t["qsl"], t["has_init"],
                                       stream=stream)
        torch.cuda.synchronize()
        return o, st

    want, side = call(), torch.cuda.Stream()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(call(side), want))
