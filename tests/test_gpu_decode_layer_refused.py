"""A refused request of the serving example keeps its length and its pages, and goes on when there is room again."""

import pytest
import torch

from tests.test_gpu_decode_layer import example  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def test_a_refused_request_keeps_its_pages(example):  # noqa: F811
    layer = example.Layer(256, heads=8, kv_heads=2, head_dim=64, experts=8, inner=128, topk=2)
    page, pages = 16, 8
    server = example.Server(layer, 3, pages, page, 6)
    g = torch.Generator(device="cuda").manual_seed(3)

    def step(new):
        x = torch.randn(sum(max(n, 0) for n in new), 256, generator=g, device="cuda").bfloat16()
        _, t = server.step(x, torch.tensor(new, dtype=torch.int32, device="cuda"), max(new))
        lens, (head, free) = server.lens.tolist(), server.ring_state.tolist()
        table, ring = server.block_table.tolist(), server.free_ring.tolist()
        held = [table[r][b] for r in range(3) for b in range(-(-lens[r] // page))]
        assert sorted(held + [ring[(head + i) % pages] for i in range(free)]) == list(range(pages))
        return t.tables.seq_lens.tolist(), lens

    assert step([48, 30, 32]) == ([48, 30, 32], [48, 30, 32])  # 7 of 8 pages
    assert step([1, 1, 1]) == ([49, 31, -1], [49, 31, 32])     # the last page goes to request 0
    assert step([1, 1, 1]) == ([50, 32, -1], [50, 32, 32])
    assert step([-1, 1, 1]) == ([0, -1, -1], [0, 32, 32])      # pages given back are there in the next step
    assert step([0, 1, 1]) == ([0, 33, 33], [0, 33, 33])
