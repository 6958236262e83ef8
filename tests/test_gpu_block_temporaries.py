"""Arguments that nobody but the call holds (a fresh copy of a bias, a sum as residual) live until the kernel is launched: the
tensors that the binding makes do not get their memory."""

import pytest
import torch

from tests import test_gpu_linear as linear
from tests.test_gpu_linear import m  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,N", [(1, 64), (3, 128), (7, 640), (40, 256), (300, 500)])
@pytest.mark.parametrize("f32", [False, True])
def test_linear(m, T, N, f32):  # noqa: F811
    p = linear.problem(T, 96, N, bias=True, residual=True, f32=f32, seed=1)
    dt = torch.float32 if f32 else torch.bfloat16
    for _ in range(3):
        torch.cuda.empty_cache()
        out = m.linear_a16w4_mxfp4(linear.on_gpu(p["x"]), torch.from_numpy(p["w"]).cuda(), torch.from_numpy(p["s"]).cuda(),
                                   bias=p["b"].cuda().clone(), residual=p["r"].cuda() * 1, out_dtype=dt)
        linear.check(p, out)


@pytest.mark.parametrize("q", [True, False])
def test_rotation(m, q):  # noqa: F811
    c = m.KvCacheMxfp4(4, 16, 2, 64)
    x = torch.randn(7, 4, 64, device="cuda").bfloat16()
    k = torch.randn(7, 2, 64, device="cuda").bfloat16()
    at = torch.arange(7, dtype=torch.int32, device="cuda")
    table = torch.randn(16, 64, device="cuda")
    want = m.kv_append_rope_mxfp4(c, x if q else None, k, k, at, at, table)
    data = m.kv_gather_mxfp4(c, at)
    for _ in range(3):
        torch.cuda.empty_cache()
        got = m.kv_append_rope_mxfp4(c, x * 1 if q else None, k * 1, k * 1, at * 1, at * 1, table * 1)
        assert got is None and want is None or torch.equal(got, want)
        assert all(torch.equal(a, b) for a, b in zip(m.kv_gather_mxfp4(c, at * 1), data))
