"""The give-up path of the linear layer's and the shared prefix's bounded waits, run on the GPU without a fault.

The wait hook (moe_set_wait_limit) gives the next call a 1 ms limit and makes one of its waits expect an arrival more than
will come (a full stage of the linear layer's tensor-core kernel, a chunk of x of its kernel for few rows, a tile's weights or a record of the attention's), so the
real wait code runs out: the kernels must record MOE_STATUS_WAIT_TIMEOUT, stop and return, and the next calls on the
workspace are right."""

import ctypes
import time

import numpy as np
import pytest
import torch

from tests import test_gpu_kv_shared as shared, test_gpu_linear as linear
from tests.test_gpu_linear import m  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def give_up(m, call, status, good):  # noqa: F811
    good(call())
    assert status() == 0
    for _ in range(2):
        assert m._native.load().moe_set_wait_limit(ctypes.c_uint64(1_000_000), 1) == 0
        t0 = time.perf_counter()
        call()  # the outputs are invalid
        assert time.perf_counter() - t0 < 1.5  # the 1 ms limit, not the 2 s default, ended the waits
        assert status() == m.MOE_STATUS_WAIT_TIMEOUT
        for _ in range(2):
            good(call())
        assert status() == 0


# few tiles (the first and the last), many: several tiles a pair of CTAs, K split in two and in three
@pytest.mark.parametrize("T,K,N", [(64, 256, 100), (700, 512, 7000), (300, 1600, 6200), (300, 2400, 4000), (40, 3200, 600)])
def test_linear(m, T, K, N):  # noqa: F811
    check_linear(m, T, K, N, None)


def check_linear(m, T, K, N, act):  # noqa: F811
    p = linear.problem(T, K, N, act=act, bias=True, seed=1)
    x, w, s, b = linear.on_gpu(p["x"]), torch.from_numpy(p["w"]).cuda(), torch.from_numpy(p["s"]).cuda(), p["b"].cuda()
    ws = torch.zeros(m.linear_workspace_bytes(T, N, K), dtype=torch.uint8, device="cuda")
    want = []

    def call():
        out = m.linear_a16w4_mxfp4(x, w, s, bias=b, act=act, workspace=ws)
        torch.cuda.synchronize()
        return out

    def good(out):
        if not want:
            linear.check(p, out)
            want.append(out)
        assert torch.equal(out, want[0])

    give_up(m, call, lambda: m.linear_read_status(ws), good)


# tensor cores: more than one wave of small tiles, K split in four and in two, not split
@pytest.mark.parametrize("T,K,N", [(40, 3200, 4860), (64, 512, 9000), (700, 256, 300)])
def test_linear_tiles(m, T, K, N):  # noqa: F811
    check_linear(m, T, K, N, "silu")


# streamed: a cluster, one chunk, more chunks than a warp's ring, partial ones, tiles of tokens
@pytest.mark.parametrize("T,K,N,act", [(32, 1600, 600, None), (20, 96, 4000, None), (17, 5152, 9000, "silu"), (25, 4096, 700, "swiglu"),
                                       (100, 4000, 290, "gelu")])
def test_linear_few_rows(m, T, K, N, act):  # noqa: F811
    check_linear(m, T, K, N, act)


# (``tail``: entries of the shared table past the prefix; with many the prefix goes to the tensor cores)
@pytest.mark.parametrize("P,R,H,G,D,tail", [(700, 40, 2, 4, 64, 0), (500, 3, 2, 4, 128, 0), (300, 60, 4, 7, 128, 0),
                                            (700, 80, 2, 4, 64, 4000), (300, 60, 4, 7, 128, 4000)])
def test_shared(m, P, R, H, G, D, tail):  # noqa: F811
    p = shared.problem(P, [30] * R, [1] * R, H, G, D, 32, seed=2, extra=1)
    p["shared"] = np.concatenate([p["shared"], np.zeros(tail, np.int32)])
    c = m.KvCacheMxfp4(p["pages"], 32, H, D, data=torch.from_numpy(p["data"]).cuda())
    i32, q = shared.i32, p["q"].cuda()
    args = (i32(p["shared"]), i32([P]), i32(p["table"]), i32(p["lens"]), i32(p["start"]), 1)
    ws = torch.zeros(m.attention_shared_workspace_bytes(c, R, R, H * G, p["table"].shape[1], 1, len(p["shared"])),
                     dtype=torch.uint8, device="cuda")

    def call():
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        m.attention_kv_mxfp4_shared(q, c, *args, scale=0.1, out=out, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        return out, lse

    give_up(m, call, lambda: m.attention_read_status(ws), lambda r: shared.check(p, *r, scale=0.1))
