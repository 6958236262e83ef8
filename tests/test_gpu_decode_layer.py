"""The operators together, as a serving loop uses them (examples/decode_layer.py), stage by stage against the oracle:
prompts and decoding requests in one step, a request that ends, its pages taken by the next."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import kv_cache as ref, moe as moe_ref, route
from tests.tolerance import assert_moe_close

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mxfp4_weight_only_gb300 import build

    build.build()
    spec = importlib.util.spec_from_file_location("decode_layer", os.path.join(ROOT, "examples", "decode_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def test_serving_steps_match_the_oracle(example):
    layer = example.Layer(256, heads=8, kv_heads=2, head_dim=64, experts=8, inner=128, topk=2)
    page, blocks, pages = 16, 24, 60
    server = example.Server(layer, 5, pages, page, blocks)
    server.cache.data.zero_()
    table = np.full((5, blocks), -1, np.int32)
    ring, state, lens = np.arange(pages, dtype=np.int32), np.array([0, pages], np.int32), np.zeros(5, np.int32)
    data = np.zeros(tuple(server.cache.data.shape), np.uint8)
    g = torch.Generator(device="cuda").manual_seed(3)
    # prompts (one long enough for the tensor-core kernel); decoding beside a late
    # prompt; a request ends; its pages are taken; all decode
    steps = [[300, 17, 1, 200, 0], [1, 1, 1, 1, 33], [-1, 1, 1, 1, 1], [250, 1, 4, 1, 1], [1, 1, 1, 1, 1]]
    for new in steps:
        N = sum(max(n, 0) for n in new)
        x = torch.randn(N, 256, generator=g, device="cuda").bfloat16()
        _, t = server.step(x, torch.tensor(new, dtype=torch.int32, device="cuda"), max(new))
        # tables
        seq, start, slots, pos, state = ref.page_tables(lens, np.array(new), table, ring, state, page, N)
        assert (seq >= 0).all()
        for got, want in ((t.tables.seq_lens, seq), (t.tables.query_start, start), (t.tables.slots, slots),
                          (t.tables.positions, pos), (server.lens, seq), (server.ring_state, state),
                          (server.free_ring, ring)):
            assert np.array_equal(got.cpu().numpy(), want)
        for r in range(5):
            used = -(-int(seq[r]) // page)
            assert np.array_equal(server.block_table[r, :used].cpu().numpy(), table[r, :used])
        # the cache
        kc, ks = ref.quantize(t.k.float().cpu().numpy())
        vc, vs = ref.quantize(t.v.float().cpu().numpy())
        for i in range(N):
            for h in range(2):
                ref.write(data, slots[i], h, kc[i, h], ks[i, h], vc[i, h], vs[i, h])
        assert np.array_equal(server.cache.data.cpu().numpy(), data)
        # attention: the bound of the attention's own tests
        want, _, spread, size = ref.attention(t.q.float().cpu().numpy(), data, table, seq, start, 64 ** -0.5)
        bound = ((2.0 ** -9 + 2.0 ** -13) * np.abs(want) +
                 (2.0 ** -9 + 2.0 ** -13 + 2 * 64 * 2.0 ** -24 * size[..., None]) * spread)
        assert (np.abs(t.attn.double().cpu().numpy() - want) <= bound).all()
        # router and experts
        logits = (t.hidden @ layer.router.T).float()
        ids, w = route.router_topk(logits.cpu().numpy(), 2)
        assert np.array_equal(t.ids.cpu().numpy(), ids) and np.allclose(t.weights.cpu().numpy(), w, rtol=1e-5)
        assert_moe_close(t.moe.double().cpu().numpy(),
                         moe_ref.moe_forward(bits(t.hidden), ids, w, layer.w13.cpu().numpy(), layer.s13.cpu().numpy(),
                                             layer.w2.cpu().numpy(), layer.s2.cpu().numpy()))
        lens = seq


def test_steps_replay_in_a_graph(example):
    layer = example.Layer(256, heads=8, kv_heads=2, head_dim=64, experts=8, inner=128, topk=2)
    runs = []
    for captured in (False, True):
        server = example.Server(layer, 3, 40, 16, 12)
        g = torch.Generator(device="cuda").manual_seed(5)
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
        runs.append((torch.stack(outs), server.lens.clone(), server.block_table.clone()))
    for a, b in zip(*runs):
        assert torch.equal(a, b)
    assert runs[0][1].tolist() == [71, 60, 22]
