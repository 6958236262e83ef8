"""A decoder layer behind a shared prefix: every request of a batch continues the same system prompt.

    python examples/prefix_layer.py [--requests 64] [--prefix 8192] [--prompt 100] [--new 64]

Random weights and random hidden states.  The prefix runs through the layer once; its keys and values stay on
pages of their own, which every request reads.  A step, for any mix of prompts and decoding requests:

    kv_page_tables             request lengths -> block table, slots, positions (the requests' own tokens)
    linear_a16w4_mxfp4         queries, keys and values, with bias
    kv_append_rope_mxfp4       rotated by their positions after the prefix, keys and values to their slots
    attention_kv_mxfp4_shared  the prefix, read once for the batch, and each request's own keys
    linear_a16w4_mxfp4         output projection, added to the residual stream
    moe_router_topk, moe_a16w4_mxfp4, and a shared expert of two more linear layers

All requests' prompts run in a first step, the decoding steps as one CUDA graph.
"""

import argparse
import os
import sys
from typing import NamedTuple

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mxfp4_weight_only_gb300 as m  # noqa: E402

i32 = dict(dtype=torch.int32, device="cuda")


class StepTrace(NamedTuple):
    tables: m.PageTables
    qkv: torch.Tensor
    q: torch.Tensor
    attn: torch.Tensor
    hidden: torch.Tensor  # after attention: the experts' input
    moe: torch.Tensor
    gated: torch.Tensor   # the shared expert's first half


class Layer:
    """Weights of one layer, all MXFP4 but the router's, and the positions' cosines and sines."""

    def __init__(self, hidden, heads, kv_heads, head_dim, experts, inner, topk, positions, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def mxfp4(*shape):
            # random codes; scale bytes of a row of values of about cols ** -0.5
            e = 127 - (shape[-1] - 1).bit_length() // 2 - 2
            return (torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=g, device="cuda", dtype=torch.uint8),
                    torch.randint(e, e + 2, (*shape[:-1], shape[-1] // 32), generator=g, device="cuda", dtype=torch.uint8))

        self.heads, self.kv_heads, self.head_dim, self.topk = heads, kv_heads, head_dim, topk
        self.wqkv, self.sqkv = mxfp4((heads + 2 * kv_heads) * head_dim, hidden)
        self.bqkv = (0.1 * torch.randn((heads + 2 * kv_heads) * head_dim, generator=g, device="cuda")).bfloat16()
        self.wo, self.so = mxfp4(hidden, heads * head_dim)
        self.router = (torch.randn(experts, hidden, generator=g, device="cuda") * hidden ** -0.5).bfloat16()
        self.w13, self.s13 = mxfp4(experts, 2 * inner, hidden)
        self.w2, self.s2 = mxfp4(experts, hidden, inner)
        self.shared13, self.shared_s13 = mxfp4(2 * inner, hidden)
        self.shared2, self.shared_s2 = mxfp4(hidden, inner)
        f = 10000.0 ** (-torch.arange(0, head_dim, 2, device="cuda", dtype=torch.float64) / head_dim)
        angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * f
        self.cos_sin = torch.cat((angle.cos(), angle.sin()), 1).float()
        # (its status word says when a wait ran out; the size does not depend on the rows)
        self.work = torch.zeros(max(m.linear_workspace_bytes(1, w.shape[0], 2 * w.shape[1]) for w in (
            self.wqkv, self.wo, self.shared13, self.shared2)), dtype=torch.uint8, device="cuda")

    def linear(self, x, w, s, **kw):
        return m.linear_a16w4_mxfp4(x, w, s, workspace=self.work, **kw)

    def project(self, x):
        """Queries, keys and values of x [N, hidden], slices of one [N, heads, head_dim] tensor."""
        qkv = self.linear(x, self.wqkv, self.sqkv, bias=self.bqkv).view(len(x), -1, self.head_dim)
        return qkv, qkv[:, :self.heads], qkv[:, self.heads:-self.kv_heads], qkv[:, -self.kv_heads:]

    def experts(self, hidden):
        """The routed experts and the shared one, added to the residual stream."""
        ids, weights = m.moe_router_topk((hidden @ self.router.T).float(), self.topk)
        moe = m.moe_a16w4_mxfp4(hidden, ids, weights, self.w13, self.s13, self.w2, self.s2)
        gated = self.linear(hidden, self.shared13, self.shared_s13, act="swiglu")
        return self.linear(gated, self.shared2, self.shared_s2, residual=hidden + moe), moe, gated


class Server:
    """One layer's cache, the prefix in it and the requests that continue it."""

    def __init__(self, layer, requests, pages, page_size, max_blocks, prefix):
        """``prefix`` bf16 [tokens, hidden]; ``pages``: for the requests, the prefix's come on top."""
        self.layer = layer
        P, first = len(prefix), -(-len(prefix) // page_size)
        self.cache = m.KvCacheMxfp4(first + pages, page_size, layer.kv_heads, layer.head_dim)
        self.shared_table = torch.arange(first, **i32)
        self.shared_len, self.prefix_len = torch.tensor([P], **i32), P
        self.block_table = torch.full((requests, max_blocks), -1, **i32)
        self.free_ring = torch.arange(first, first + pages, **i32)
        self.ring_state = torch.tensor([0, pages], **i32)
        self.lens = torch.zeros(requests, **i32)
        need = m.attention_workspace_bytes(self.cache, 1, P, layer.heads, first, P)
        self.workspace = torch.zeros(need, dtype=torch.uint8, device="cuda")
        # the prefix runs as one prompt on its own pages
        _, q, k, v = layer.project(prefix)
        at = torch.arange(P, **i32)
        q = m.kv_append_rope_mxfp4(self.cache, q, k, v, at, at, layer.cos_sin)
        start = torch.tensor([0, P], **i32)
        attn = m.attention_kv_mxfp4(q, self.cache, self.shared_table[None], self.shared_len, start, P,
                                    workspace=self.workspace)
        hidden = layer.linear(attn.flatten(1), layer.wo, layer.so, residual=prefix)
        self.prefix_out = layer.experts(hidden)[0]  # what the next layer's prefix would be

    def check(self):
        """Raises if a wait of an attention or a linear layer since the last check ran out (its outputs are invalid)."""
        if m.attention_read_status(self.workspace):
            raise RuntimeError("an attention kernel gave up waiting")
        if m.linear_read_status(self.layer.work):
            raise RuntimeError("a linear layer's kernel gave up waiting")

    def step(self, x, new_lens, max_q_len):
        """``x`` bf16 [tokens, hidden], the tokens of ``new_lens`` (int32 [requests], -1: finished) in order."""
        L, N = self.layer, x.shape[0]
        tables = m.kv_page_tables(self.lens, new_lens, self.block_table, self.free_ring, self.ring_state,
                                  self.cache.page_size, N)
        qkv, q, k, v = L.project(x)
        q = m.kv_append_rope_mxfp4(self.cache, q, k, v, tables.positions, tables.slots, L.cos_sin,
                                   position_offset=self.prefix_len)
        need = m.attention_shared_workspace_bytes(self.cache, len(self.lens), N, L.heads, self.block_table.shape[1],
                                                  max_q_len, len(self.shared_table))
        if self.workspace.numel() < need:
            self.check()
            self.workspace = torch.zeros(need, dtype=torch.uint8, device="cuda")
        attn = m.attention_kv_mxfp4_shared(q, self.cache, self.shared_table, self.shared_len, self.block_table,
                                           tables.seq_lens, tables.query_start, max_q_len, workspace=self.workspace)
        hidden = L.linear(attn.flatten(1), L.wo, L.so, residual=x)
        y, moe, gated = L.experts(hidden)
        # a refused request (-1) keeps its length and pages: the caller gives its tokens again
        self.lens.copy_(torch.where(tables.seq_lens < 0, self.lens, tables.seq_lens))
        self.ring_state.copy_(tables.ring_state)
        return y, StepTrace(tables, qkv, q, attn, hidden, moe, gated)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=64)
    ap.add_argument("--prefix", type=int, default=8192)
    ap.add_argument("--prompt", type=int, default=100)
    ap.add_argument("--new", type=int, default=64)
    args = ap.parse_args()
    hidden, page = 3584, 64
    own = args.prompt + args.new + 2
    layer = Layer(hidden, heads=28, kv_heads=4, head_dim=128, experts=32, inner=1024, topk=4, positions=args.prefix + own)
    g = torch.Generator(device="cuda").manual_seed(1)
    prefix = torch.randn(args.prefix, hidden, generator=g, device="cuda").bfloat16()
    blocks, R = -(-own // page), args.requests
    server = Server(layer, R, R * blocks, page, blocks, prefix)
    x = torch.randn(R * args.prompt, hidden, generator=g, device="cuda").bfloat16()
    y, _ = server.step(x, torch.full((R,), args.prompt, **i32), args.prompt)
    state = y[args.prompt - 1::args.prompt].contiguous()  # each prompt's last token
    one = torch.ones(R, **i32)

    def decode():
        y, _ = server.step(state, one, 1)
        state.copy_(y * torch.rsqrt(y.float().square().mean(-1, keepdim=True)))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        decode()  # a first step outside the graph: libraries load
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        decode()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(args.new):
        graph.replay()
    end.record()
    end.synchronize()
    ms = begin.elapsed_time(end) / args.new
    server.check()
    lens = server.lens.cpu()
    assert (lens == args.prompt + args.new + 1).all(), lens
    assert torch.isfinite(state.float()).all() and torch.isfinite(server.prefix_out.float()).all()
    print(f"{R} requests of {args.prompt} tokens behind a prefix of {args.prefix}, {args.new} decoding steps: "
          f"{ms * 1000:.0f} us a step and layer, {server.cache.data.numel() / 2 ** 20:.0f} MiB of cache")


if __name__ == "__main__":
    main()
