"""Serving steps of one decoder layer: 4-bit KV cache, attention over it, router, MoE.

    python examples/decode_layer.py [--requests 32] [--prompt 1000] [--new 64]

Random weights of the default MoE configuration's widths and random hidden
states.  A step, for any mix of prompts and decoding requests:

    kv_page_tables        request lengths -> block table, slots, positions
    (projection, rotary)  plain PyTorch
    kv_append_mxfp4       the step's keys and values, slices of the projection, to their slots
    attention_kv_mxfp4    the step's queries over the cache
    (projection)          plain PyTorch
    moe_router_topk, moe_a16w4_mxfp4

All requests' prompts run in a first step, the decoding steps as one CUDA graph:
lengths, tables and the ring of free pages stay on the GPU.
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
    k: torch.Tensor
    v: torch.Tensor
    q: torch.Tensor
    attn: torch.Tensor
    hidden: torch.Tensor  # after attention: the MoE's input
    ids: torch.Tensor
    weights: torch.Tensor
    moe: torch.Tensor


class Layer:
    """Weights of one layer: fused q/k/v projection, output projection, router, experts."""

    def __init__(self, hidden, heads, kv_heads, head_dim, experts, inner, topk, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def bf16(*shape):
            return (torch.randn(*shape, generator=g, device="cuda") * shape[-1] ** -0.5).bfloat16()

        def mxfp4(rows, cols):
            # random codes; scale bytes of a row of values of about cols ** -0.5
            e = 127 - (cols - 1).bit_length() // 2 - 2
            return (torch.randint(0, 256, (experts, rows, cols // 2), generator=g, device="cuda", dtype=torch.uint8),
                    torch.randint(e, e + 2, (experts, rows, cols // 32), generator=g, device="cuda", dtype=torch.uint8))

        self.heads, self.kv_heads, self.head_dim, self.topk = heads, kv_heads, head_dim, topk
        self.wqkv = bf16((heads + 2 * kv_heads) * head_dim, hidden)
        self.wo = bf16(hidden, heads * head_dim)
        self.router = bf16(experts, hidden)
        self.w13, self.s13 = mxfp4(2 * inner, hidden)
        self.w2, self.s2 = mxfp4(hidden, inner)
        half = head_dim // 2
        self.freq = 10000.0 ** (-torch.arange(half, device="cuda") / half)


class Server:
    """One layer's cache and the requests in it."""

    def __init__(self, layer, requests, pages, page_size, max_blocks):
        self.layer = layer
        self.cache = m.KvCacheMxfp4(pages, page_size, layer.kv_heads, layer.head_dim)
        self.block_table = torch.full((requests, max_blocks), -1, **i32)
        self.free_ring = torch.arange(pages, **i32)
        self.ring_state = torch.tensor([0, pages], **i32)
        self.lens = torch.zeros(requests, **i32)
        self.workspace = torch.zeros(0, dtype=torch.uint8, device="cuda")

    def check(self):
        """Raises if a wait of an attention since the last check ran out (its outputs are invalid)."""
        if self.workspace.numel() and m.attention_read_status(self.workspace):
            raise RuntimeError("an attention kernel gave up waiting")

    def rotary(self, x, positions):
        angle = positions.clamp(min=0).float()[:, None, None] * self.layer.freq
        a, b = x.float().chunk(2, dim=-1)
        return torch.cat((a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()), -1).to(x.dtype)

    def step(self, x, new_lens, max_q_len):
        """``x`` bf16 [tokens, hidden], the tokens of ``new_lens`` (int32 [requests], -1: finished) in order."""
        L, N = self.layer, x.shape[0]
        tables = m.kv_page_tables(self.lens, new_lens, self.block_table, self.free_ring, self.ring_state,
                                  self.cache.page_size, N)
        qkv = (x @ L.wqkv.T).view(N, L.heads + 2 * L.kv_heads, L.head_dim)
        turned = self.rotary(qkv[:, :L.heads + L.kv_heads], tables.positions)
        q, k = turned[:, :L.heads], turned[:, L.heads:]
        v = qkv[:, L.heads + L.kv_heads:]
        m.kv_append_mxfp4(self.cache, k, v, tables.slots)
        need = m.attention_workspace_bytes(self.cache, len(self.lens), N, L.heads, self.block_table.shape[1], max_q_len)
        if self.workspace.numel() < need:
            self.check()
            self.workspace = torch.zeros(need, dtype=torch.uint8, device="cuda")
        attn = m.attention_kv_mxfp4(q, self.cache, self.block_table, tables.seq_lens, tables.query_start, max_q_len,
                                    workspace=self.workspace)
        hidden = x + attn.view(N, L.heads * L.head_dim) @ L.wo.T
        ids, weights = m.moe_router_topk((hidden @ L.router.T).float(), L.topk)
        moe = m.moe_a16w4_mxfp4(hidden, ids, weights, L.w13, L.s13, L.w2, L.s2)
        # a refused request (-1) keeps its length and pages: the caller gives its tokens again
        self.lens.copy_(torch.where(tables.seq_lens < 0, self.lens, tables.seq_lens))
        self.ring_state.copy_(tables.ring_state)
        return hidden + moe, StepTrace(tables, k, v, q, attn, hidden, ids, weights, moe)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=32)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--new", type=int, default=64)
    args = ap.parse_args()
    hidden, page = 3584, 64
    layer = Layer(hidden, heads=28, kv_heads=4, head_dim=128, experts=32, inner=1024, topk=4)
    blocks = -(-(args.prompt + args.new + 2) // page)
    server = Server(layer, args.requests, args.requests * blocks, page, blocks)
    R = args.requests
    g = torch.Generator(device="cuda").manual_seed(1)
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
    assert torch.isfinite(state.float()).all()
    print(f"{R} requests of {args.prompt} tokens, {args.new} decoding steps: {ms * 1000:.0f} us a step and layer, "
          f"{server.cache.data.numel() / 2 ** 20:.0f} MiB of cache")
    # one request ends: its pages go back to the ring
    done = one.clone()
    done[0] = -1
    free = int(server.ring_state[1])
    server.step(state[1:].contiguous(), done, 1)
    print(f"free pages: {free} before a request ended, {int(server.ring_state[1])} after")


if __name__ == "__main__":
    main()
