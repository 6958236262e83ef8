"""The operators together, as a serving loop behind a shared prefix uses them (examples/prefix_layer.py), stage by stage
against the oracle: the prefix, prompts and decoding requests in one step, a request that ends, its pages taken by the
next, a step replayed in a graph."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import block, kv_cache as cache_ref, kv_shared as ref, moe as moe_ref, route
from tests.tolerance import assert_moe_close

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
D, H, HEADS, PAGE, PREFIX = 64, 2, 8, 16, 300


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mxfp4_weight_only_gb300 import build

    build.build()
    spec = importlib.util.spec_from_file_location("prefix_layer", os.path.join(ROOT, "examples", "prefix_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def num(t):
    return t.double().cpu().numpy()


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def close(got, x, w, s, **kw):
    """A linear layer's result, by the bound of its own tests."""
    want, slack = block.linear(num(x), w.cpu().numpy(), s.cpu().numpy(), **kw)
    K, a = x.shape[1], 2.0 ** -18 if kw.get("act") else 0.0
    bound = ((K + 1) * 2.0 ** -23 + a) * slack + (a + 2.0 ** -23 + 2.0 ** -8) * np.abs(want)
    if kw.get("residual") is not None:
        bound = bound + 2.0 ** -23 * np.abs(kw["residual"])
    assert (np.abs(num(got) - want) <= bound).all()


def rotated(layer, rows, positions):
    """float32 rows [N, heads, D] as the kernel turns them."""
    cs = layer.cos_sin.cpu().numpy()
    return np.stack([block.rotate(r, cs[p]) for r, p in zip(rows.float().cpu().numpy(), positions)])


def write(data, layer, qkv, positions, slots):
    k = rotated(layer, qkv[:, HEADS:-H], positions)
    kc, ks = cache_ref.quantize(k)
    vc, vs = cache_ref.quantize(qkv[:, -H:].float().cpu().numpy())
    for i, slot in enumerate(slots):
        for h in range(H):
            cache_ref.write(data, slot, h, kc[i, h], ks[i, h], vc[i, h], vs[i, h])


def make(example, requests=4, pages=40, blocks=14):
    layer = example.Layer(256, heads=HEADS, kv_heads=H, head_dim=D, experts=8, inner=128, topk=2, positions=1000)
    g = torch.Generator(device="cuda").manual_seed(3)
    prefix = torch.randn(PREFIX, 256, generator=g, device="cuda").bfloat16()
    return layer, example.Server(layer, requests, pages, PAGE, blocks, prefix), prefix, g


def test_serving_steps_match_the_oracle(example):
    layer, server, prefix, g = make(example)
    first = -(-PREFIX // PAGE)
    # the prefix's keys and values, written once
    data = np.zeros(tuple(server.cache.data.shape), np.uint8)
    qkv = layer.project(prefix)[0]
    close(qkv.flatten(1), prefix, layer.wqkv, layer.sqkv, bias=num(layer.bqkv))
    write(data, layer, qkv, range(PREFIX), range(PREFIX))
    used = np.zeros(data.shape, bool)
    mark = np.full((PREFIX, H, D // 2), 1, np.uint8)
    ones = np.zeros(data.shape, np.uint8)
    for i in range(PREFIX):
        for h in range(H):
            cache_ref.write(ones, i, h, mark[i, h], mark[i, h, : D // 32], mark[i, h], mark[i, h, : D // 32])
    used = ones == 1
    assert np.array_equal(server.cache.data.cpu().numpy()[used], data[used])
    server.cache.data.copy_(torch.from_numpy(data))
    table = np.full((4, 14), -1, np.int32)
    ring, state, lens = np.arange(first, first + 40, dtype=np.int32), np.array([0, 40], np.int32), np.zeros(4, np.int32)
    for new in ([90, 17, 1, 0], [1, 1, 1, 60], [-1, 1, 1, 1], [120, 1, 4, 1], [1, 1, 1, 1]):
        N = sum(max(n, 0) for n in new)
        x = torch.randn(N, 256, generator=g, device="cuda").bfloat16()
        y, t = server.step(x, torch.tensor(new, dtype=torch.int32, device="cuda"), max(new))
        server.check()
        seq, start, slots, pos, state = cache_ref.page_tables(lens, np.array(new), table, ring, state, PAGE, N)
        assert (seq >= 0).all() and np.array_equal(t.tables.seq_lens.cpu().numpy(), seq)
        close(t.qkv.flatten(1), x, layer.wqkv, layer.sqkv, bias=num(layer.bqkv))
        # queries and cache: exact
        assert torch.equal(t.q.cpu(), torch.from_numpy(rotated(layer, t.qkv[:, :HEADS], pos + PREFIX)).bfloat16())
        write(data, layer, t.qkv, pos + PREFIX, slots)
        assert np.array_equal(server.cache.data.cpu().numpy(), data)
        # attention: the bound of its own tests (a finished request has no rows)
        want, _, spread, size = ref.attention(num(t.q), data, server.shared_table.cpu().numpy(), PREFIX, table, seq, start, D ** -0.5)
        bound = ((2.0 ** -8 + 2.0 ** -13) * np.abs(want) +
                 (2.0 ** -9 + 2.0 ** -13 + 2 * (D + 2) * 2.0 ** -24 * size[..., None]) * spread)
        assert (np.abs(num(t.attn) - want) <= bound).all()
        close(t.hidden, t.attn.flatten(1), layer.wo, layer.so, residual=num(x))
        ids, w = route.router_topk((t.hidden @ layer.router.T).float().cpu().numpy(), 2)
        assert_moe_close(num(t.moe), moe_ref.moe_forward(bits(t.hidden), ids, w, layer.w13.cpu().numpy(), layer.s13.cpu().numpy(),
                                                         layer.w2.cpu().numpy(), layer.s2.cpu().numpy()))
        close(t.gated, t.hidden, layer.shared13, layer.shared_s13, act="swiglu")
        close(y, t.gated, layer.shared2, layer.shared_s2, residual=num(t.hidden + t.moe))
        lens = seq


def test_steps_replay_in_a_graph(example):
    runs = []
    for captured in (False, True):
        _, server, _, g = make(example, requests=3)
        x = torch.randn(90, 256, generator=g, device="cuda").bfloat16()
        server.step(x, torch.tensor([50, 39, 1], dtype=torch.int32, device="cuda"), 50)
        one = torch.ones(3, dtype=torch.int32, device="cuda")
        tok = torch.randn(3, 256, generator=g, device="cuda").bfloat16()
        y, _ = server.step(tok, one, 1)
        outs = []
        if captured:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                y, _ = server.step(tok, one, 1)
            for _ in range(20):
                graph.replay()
                outs.append(y.clone())
        else:
            for _ in range(20):
                outs.append(server.step(tok, one, 1)[0])
        server.check()
        runs.append((torch.stack(outs), server.lens.clone(), server.block_table.clone()))
    for a, b in zip(*runs):
        assert torch.equal(a, b)
    assert runs[0][1].tolist() == [71, 60, 22]
