"""The limit of the linear layer's waits bounds a stage, not the call: one of many tiles a pair of CTAs runs longer than the
limit, each of its waits for a few microseconds, and none runs out."""

import ctypes

import pytest
import torch

from tests.test_gpu_linear import m  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def test_a_call_longer_than_the_limit(m):  # noqa: F811
    T, K, N = 32768, 512, 131072
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    w = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, generator=g, device="cuda")
    s = torch.randint(115, 122, (N, K // 32), dtype=torch.uint8, generator=g, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    out = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    m.linear_a16w4_mxfp4(x, w, s, out=out, workspace=ws)
    first = out[::97].clone()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    assert m._native.load().moe_set_wait_limit(ctypes.c_uint64(500_000), 0) == 0
    begin.record()
    m.linear_a16w4_mxfp4(x, w, s, out=out, workspace=ws)
    end.record()
    assert m.linear_read_status(ws) == 0
    assert begin.elapsed_time(end) > 1.0  # ms: twice the limit, a hundred tiles a pair of CTAs and more
    assert torch.equal(out[::97], first)
