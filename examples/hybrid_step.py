"""An engine step of a small hybrid stack: Gated DeltaNet layers and one
full-attention layer, decode rows and prompt chunks in one batch.

    python examples/hybrid_step.py

The step's lengths, free list, block table and positions live on the GPU and
gdn_build_step_tables works on them there, so that a decode step is one HIP
graph that is replayed as it is: no length comes back to the host.  Weights are
random, and hidden states stand for the embedding and the feed-forward blocks.
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_token_amd as gdn  # noqa: E402

HIDDEN, EPS = 2560, 1e-6
HK, HV, D = 16, 32, 128                    # Gated DeltaNet: q/k heads, v heads, their size
C = (2 * HK + HV) * D                      # conv channels: q | k | v
AQ, AK, AD, ROT = 16, 4, 256, 64           # attention: q heads, kv heads, their size, rotated elements
PAGE = 16
LAYERS = ("delta", "delta", "delta", "attention")
BF16 = torch.bfloat16


class HybridStack:
    def __init__(self, num_requests, max_len, seed=0, device="cuda"):
        gen = torch.Generator(device).manual_seed(seed)

        def normal(*shape, std=1.0, dtype=BF16):
            return (std * torch.randn(*shape, generator=gen, device=device)).to(dtype)

        self.max_len, S = max_len, num_requests
        columns = -(-max_len // PAGE)
        pages = S * columns
        i32 = dict(dtype=torch.int32, device=device)
        self.context_lens = torch.zeros(S, **i32)
        self.free_pages = torch.randperm(pages, generator=gen, device=device).to(torch.int32)
        self.num_free = torch.full((1,), pages, **i32)
        self.block_table = torch.full((S, columns), -1, **i32)
        self.slots = torch.arange(S, **i32)                      # of the recurrent states
        frequencies, self.rope_scale = gdn.gdn_rope_frequencies(ROT, 1e7)
        self.frequencies = torch.from_numpy(frequencies).to(device)
        self.zero = torch.zeros(1, HIDDEN, dtype=BF16, device=device)
        self.norms = [normal(HIDDEN, std=0.1) for _ in range(len(LAYERS) + 1)]        # about one: weight_offset 1
        self.layers = []
        for kind in LAYERS:
            p = {}
            if kind == "delta":
                p["w_in"] = normal(HIDDEN, C + HV * D + 2 * HV, std=HIDDEN ** -0.5)   # q | k | v | gate | beta | decay
                p["w_out"] = normal(HV * D, HIDDEN, std=(HV * D) ** -0.5)
                p["conv"], p["norm"] = normal(C, 4, std=0.5), normal(D, std=0.1)
                p["decay"], p["bias"] = normal(HV, dtype=torch.float32).exp(), normal(HV, dtype=torch.float32)
                p["conv_state"] = torch.zeros(S, 3, C, dtype=BF16, device=device)
                p["state"] = torch.zeros(S, HV, D, D, device=device)
            else:
                p["w_in"] = normal(HIDDEN, (2 * AQ + 2 * AK) * AD, std=HIDDEN ** -0.5)        # q | k | v | gate
                p["w_out"] = normal(AQ * AD, HIDDEN, std=(AQ * AD) ** -0.5)
                p["q_norm"], p["k_norm"] = normal(AD, std=0.1), normal(AD, std=0.1)
                code = dict(dtype=torch.uint8, device=device)
                p["k_cache"] = torch.zeros(pages, AK, PAGE, AD, **code).view(torch.float8_e4m3fn)
                p["v_cache"] = torch.zeros(pages, AK, AD, PAGE, **code).view(torch.float8_e4m3fn)
                p["k_scale"] = torch.zeros(pages, AK, device=device)
                p["v_scale"] = torch.zeros(pages, AK, device=device)
            self.layers.append(p)

    def delta(self, p, h, t, decode):
        T = h.shape[0]
        u = h @ p["w_in"]
        x, gate = u[:, :C], u[:, C:C + HV * D].view(T, HV, D)
        beta = torch.sigmoid(u[:, C + HV * D:C + HV * D + HV].float())
        g = -p["decay"] * torch.nn.functional.softplus(u[:, C + HV * D + HV:].float() + p["bias"])
        o = torch.empty(T, HV, D, dtype=BF16, device=h.device)
        if decode:
            gdn.gdn_fused_conv_decode(x, p["conv"], None, p["conv_state"], g, beta, p["state"], self.slots, o, HK, D,
                                      scale=D ** -0.5)
        else:
            y = torch.empty(T, C, dtype=BF16, device=h.device)
            gdn.gdn_causal_conv1d_varlen(x, p["conv"], None, p["conv_state"], t["query_start_loc"], self.slots,
                                         t["has_context"], t["chunks"], y)
            q, k, v = y[:, :HK * D], y[:, HK * D:2 * HK * D], y[:, 2 * HK * D:]
            gdn.gdn_chunk_gated_delta_rule(q.view(T, HK, D), k.view(T, HK, D), v.view(T, HV, D), g, beta, p["state"],
                                           self.slots, o, t["query_start_loc"], t["has_context"], scale=D ** -0.5)
        gdn.gdn_gated_rms_norm(o, p["norm"], o, gate=gate, eps=EPS, weight_offset=1.0)
        return o.view(T, HV * D) @ p["w_out"]

    def attention(self, p, h, t, max_seq_len):
        T = h.shape[0]
        u = (h @ p["w_in"]).view(T, 2 * AQ + 2 * AK, AD)
        q, k, v, gate = u[:, :AQ], u[:, AQ:AQ + AK], u[:, AQ + AK:AQ + 2 * AK], u[:, AQ + 2 * AK:]
        gdn.gdn_gated_rms_norm(q, p["q_norm"], q, eps=EPS, weight_offset=1.0)
        gdn.gdn_gated_rms_norm(k, p["k_norm"], k, eps=EPS, weight_offset=1.0)
        cache = (p["k_cache"], p["v_cache"], p["k_scale"], p["v_scale"])
        gdn.gdn_rope_append_kv8(q, k, v, t["positions"], t["slot_mapping"], self.frequencies, q, *cache,
                                rope_scale=self.rope_scale)
        o = torch.empty(T, AQ, AD, dtype=BF16, device=h.device)
        gdn.gdn_paged_attention_kv8(q, *cache, self.block_table, t["seq_lens"], t["query_start_loc"], o, max_seq_len,
                                    AD ** -0.5)
        return (o * torch.sigmoid(gate)).view(T, AQ * AD) @ p["w_out"]

    def step(self, x, query_lens, max_seq_len, decode=False):
        """Hidden states x [T][HIDDEN] of the step's new tokens, query_lens[s] of
        request s in order, through every layer; ``decode``: one token each.
        ``max_seq_len``: the longest request after the step, or a bound."""
        T, S, dev = x.shape[0], query_lens.shape[0], x.device
        i32 = dict(dtype=torch.int32, device=dev)
        t = {"query_start_loc": torch.empty(S + 1, **i32), "seq_lens": torch.empty(S, **i32),
             "positions": torch.empty(T, **i32), "slot_mapping": torch.empty(T, dtype=torch.int64, device=dev),
             "counts": torch.empty(4, **i32),
             "chunks": None if decode else torch.empty(T // 8 + S, 2, **i32),
             "has_context": (self.context_lens > 0).to(torch.uint8)}
        gdn.gdn_build_step_tables(self.context_lens, query_lens, self.free_pages, self.num_free, self.block_table, PAGE,
                                  t["query_start_loc"], t["seq_lens"], t["positions"], t["slot_mapping"], t["counts"],
                                  t["chunks"])
        residual, h = torch.empty_like(x), torch.empty_like(x)
        gdn.gdn_residual_rms_norm(x, self.zero.expand(T, HIDDEN).contiguous(), self.norms[0], residual, h, eps=EPS,
                                  weight_offset=1.0)
        for kind, p, norm in zip(LAYERS, self.layers, self.norms[1:]):
            u = self.delta(p, h, t, decode) if kind == "delta" else self.attention(p, h, t, max_seq_len)
            gdn.gdn_residual_rms_norm(u, residual, norm, residual, h, eps=EPS, weight_offset=1.0)
        self.context_lens.copy_(t["seq_lens"])
        self.num_free.sub_(t["counts"][2:3])
        return h, t


def main():
    lens, new = [300, 1, 517, 64], 32
    stack = HybridStack(len(lens), max_len=1024)
    gen = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(sum(lens), HIDDEN, generator=gen, device="cuda").to(BF16)
    h, t = stack.step(x, torch.tensor(lens, dtype=torch.int32, device="cuda"), max(lens))
    print("prompts of %s tokens: %d pages taken, %d missing" % (lens, *t["counts"][2:].tolist()))

    ends = t["query_start_loc"][1:].long() - 1
    one = torch.ones(len(lens), dtype=torch.int32, device="cuda")
    x = h[ends].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                     # a decode step outside the graph first
        h, _ = stack.step(x, one, stack.max_len, decode=True)
        x.copy_(h)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, t = stack.step(x, one, stack.max_len, decode=True)
        x.copy_(h)
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(new - 1):
        graph.replay()
    torch.cuda.synchronize()
    took = time.perf_counter() - start
    print("%d decode steps of %d requests: %.0f us a step; lengths now %s, %d pages free"
          % (new, len(lens), took / (new - 1) * 1e6, stack.context_lens.tolist(), int(stack.num_free)))
    return stack, h


if __name__ == "__main__":
    main()
