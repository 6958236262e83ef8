"""The example behind a shared prefix sees a wait of its attention or of a linear layer that ran out."""

import ctypes

import pytest
import torch

from tests.test_gpu_prefix_layer import example  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def test_a_wait_that_ran_out_is_seen(example, monkeypatch):  # noqa: F811
    m = example.m
    layer = example.Layer(256, heads=8, kv_heads=2, head_dim=64, experts=8, inner=128, topk=2, positions=400)
    prefix = torch.randn(100, 256, device="cuda").bfloat16()
    server = example.Server(layer, 3, 40, 16, 12, prefix)
    server.check()
    x = torch.randn(90, 256, device="cuda").bfloat16()
    lens = torch.tensor([50, 39, 1], dtype=torch.int32, device="cuda")
    server.step(x, lens, 50)
    server.check()

    def give_up(name):
        """The next call of ``name`` waits for what does not come."""
        real = getattr(m, name)

        def call(*a, **kw):
            monkeypatch.setattr(m, name, real)
            assert m._native.load().moe_set_wait_limit(ctypes.c_uint64(1_000_000), 1) == 0
            return real(*a, **kw)

        monkeypatch.setattr(m, name, call)

    give_up("attention_kv_mxfp4_shared")
    server.step(x, lens, 50)
    with pytest.raises(RuntimeError, match="attention"):
        server.check()
    give_up("linear_a16w4_mxfp4")  # (90 rows: a kernel that waits)
    server.step(x, lens, 50)
    with pytest.raises(RuntimeError, match="linear"):
        server.check()
    # the prefix's own
    give_up("attention_kv_mxfp4")
    late = example.Server(layer, 3, 40, 16, 12, prefix)
    with pytest.raises(RuntimeError, match="attention"):
        late.check()
    server.step(x[:3], torch.ones_like(lens), 1)
    server.check()
