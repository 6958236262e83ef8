"""The serving example sees a wait of its attention that ran out."""

import ctypes

import pytest
import torch

from tests.test_gpu_decode_layer import example  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def test_a_wait_that_ran_out_is_seen(example):  # noqa: F811
    m = example.m
    layer = example.Layer(256, heads=8, kv_heads=2, head_dim=64, experts=8, inner=128, topk=2)
    server = example.Server(layer, 3, 40, 16, 12)
    x = torch.randn(90, 256, device="cuda").bfloat16()
    lens = torch.tensor([50, 39, 1], dtype=torch.int32, device="cuda")
    server.step(x, lens, 50)
    server.check()
    assert m._native.load().moe_set_wait_limit(ctypes.c_uint64(1_000_000), 1) == 0
    server.step(x, lens, 50)
    with pytest.raises(RuntimeError, match="attention"):
        server.check()
    server.step(x[:3], torch.ones_like(lens), 1)
    server.check()
