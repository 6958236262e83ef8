"""Sizes and offsets that the C ABI's int32 does not hold: taken as they are meant or refused, never by their low 32 bits."""

import pytest
import torch

from tests import test_gpu_kv_shared as shared
from tests.test_gpu_linear import m  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

i32 = shared.i32


def test_position_offset(m):  # noqa: F811
    c = m.KvCacheMxfp4(2, 16, 1, 64)
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(3, 1, 64, generator=g, device="cuda").bfloat16() for _ in range(3))
    table = torch.randn(8, 32, generator=g, device="cuda")
    args = (c, q, k, v, i32([0, 1, -1]), i32([0, 1, 2]), table)
    near = m.kv_append_rope_mxfp4(*args)
    assert torch.isfinite(near).all()
    for far in (8, 2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 1, 2 ** 40):
        out = m.kv_append_rope_mxfp4(*args, position_offset=far)
        assert torch.isnan(out[:2]).all() and (out[2] == 0).all(), far  # past the table; padding
        assert torch.isnan(m.kv_gather_mxfp4(c, i32([0, 1]))[0]).all()
    for bad in (-1, -2 ** 31, -2 ** 32, -2 ** 32 + 1):
        with pytest.raises(m.MoeError):
            m.kv_append_rope_mxfp4(*args, position_offset=bad)


def test_max_q_len(m):  # noqa: F811
    p = shared.problem(100, [9, 4], [5, 3], 2, 4, 64, 16)
    want = shared.run(m, p)
    c = m.KvCacheMxfp4(p["pages"], 16, 2, 64, data=torch.from_numpy(p["data"]).cuda())
    q = p["q"].cuda()
    args = (q, c, i32(p["shared"]), i32([100]), i32(p["table"]), i32(p["lens"]), i32(p["start"]))
    plain = (q, c, i32(p["table"]), i32(p["lens"]), i32(p["start"]))
    ref = m.attention_kv_mxfp4(*plain, 5, scale=0.2)
    for n in (2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 3, 2 ** 40):
        assert torch.allclose(m.attention_kv_mxfp4_shared(*args, n, scale=0.2).float(), want[0].float(), rtol=2 ** -6, atol=2 ** -7)
        assert torch.allclose(m.attention_kv_mxfp4(*plain, n, scale=0.2).float(), ref.float(), rtol=2 ** -6, atol=2 ** -7)
        assert m.attention_shared_workspace_bytes(c, 2, 8, 8, p["table"].shape[1], n, len(p["shared"])) > 0
    for n in (-1, -2 ** 31, -2 ** 32, -2 ** 32 + 4):
        with pytest.raises(m.MoeError):
            m.attention_kv_mxfp4_shared(*args, n)
        with pytest.raises(m.MoeError):
            m.attention_kv_mxfp4(*plain, n)


def test_weight_sizes(m):  # noqa: F811
    # 32 rows by their low bits (nothing is read or written)
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("a weight of 2^32 rows needs 69 GB")
    N = 2 ** 32 + 32
    w = torch.empty(N, 16, dtype=torch.uint8, device="cuda")
    s = torch.empty(N, 1, dtype=torch.uint8, device="cuda")
    x = torch.zeros(1, 32, dtype=torch.bfloat16, device="cuda")
    with pytest.raises((ValueError, m.MoeError)):
        m.linear_a16w4_mxfp4(x, w, s)
    del w, s, x
    torch.cuda.empty_cache()
    # 64 columns by their low bits
    x = torch.empty(1, 2 ** 32 + 64, dtype=torch.bfloat16, device="cuda")
    w = torch.empty(1, 2 ** 31 + 32, dtype=torch.uint8, device="cuda")
    s = torch.empty(1, 2 ** 27 + 2, dtype=torch.uint8, device="cuda")
    with pytest.raises((ValueError, m.MoeError)):
        m.linear_a16w4_mxfp4(x, w, s)
    assert m.linear_workspace_bytes(2 ** 32 + 1, 64, 64) == 0 and m.linear_workspace_bytes(1, 64, 2 ** 32 + 64) == 0
    del w, s
    torch.cuda.empty_cache()
