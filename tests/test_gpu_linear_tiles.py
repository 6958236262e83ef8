"""The linear layer on an MXFP4 weight beyond two waves of 32 x 32 tiles, where tcgen05 MMAs of CTA pairs do it: rows and
columns around their tiles, depths, epilogues, addresses, values of unlike size.  The same float64 oracle and derived
bound as for smaller ones."""

import numpy as np
import pytest
import torch

from tests import test_gpu_linear as linear
from tests.test_gpu_linear import both, call, check, m, on_gpu, problem  # noqa: F401

pytestmark = pytest.mark.gpu


def rows_for(T, more=0):
    """Weight rows of the first size past two waves, and ``more``."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return 32 * (2 * sms // -(-T // 32)) + 2 + more


@pytest.mark.parametrize("T", [33, 63, 64, 65, 100, 127, 128, 129, 200, 255, 256, 257, 300, 513, 1100])
def test_rows(m, T):  # noqa: F811
    both(m, T, 256, rows_for(T), seed=1)
    both(m, T, 96, rows_for(T, 131), seed=1)


@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 480, 992, 1024, 2080, 4096, 8192])
@pytest.mark.parametrize("T", [40, 150, 300])
def test_depths(m, K, T):  # noqa: F811
    both(m, T, K, rows_for(T, 21), seed=2, bias=True)


@pytest.mark.parametrize("N", [255, 256, 257, 270, 287, 288, 289, 383, 384, 385, 500, 511, 512, 513, 767, 769, 1111])
@pytest.mark.parametrize("T", [620, 1300])
def test_columns(m, N, T):  # noqa: F811
    both(m, T, 192, N, seed=3, bias=True, residual=True)


@pytest.mark.parametrize("act", [None, "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("bias,residual,f32", [(False, False, False), (True, False, True), (False, True, True), (True, True, False)])
@pytest.mark.parametrize("T", [50, 140, 600])
def test_epilogues(m, act, bias, residual, f32, T):  # noqa: F811
    both(m, T, 288, rows_for(T, 154), act=act, bias=bias, residual=residual, f32=f32, seed=4)
    both(m, T, 512, rows_for(T, 30), act=act, bias=bias, residual=residual, f32=f32, seed=5)


@pytest.mark.parametrize("T", [50, 300])
@pytest.mark.parametrize("K", [32, 96, 160, 2080])
@pytest.mark.parametrize("skip", [1, 2, 3])
def test_scales_at_any_address(m, T, K, skip):  # noqa: F811
    p = problem(T, K, rows_for(T), seed=6)
    tall = torch.full((p["N"] + 2 * skip, K // 32), 255, dtype=torch.uint8, device="cuda")
    s = tall[skip: skip + p["N"]]
    s.copy_(torch.from_numpy(p["s"]))
    check(p, m.linear_a16w4_mxfp4(on_gpu(p["x"]), torch.from_numpy(p["w"]).cuda(), s))


@pytest.mark.parametrize("T", [130, 520])
@pytest.mark.parametrize("pad", [1, 3, 8])
def test_strided_rows(m, T, pad):  # noqa: F811
    for act, f32 in ((None, False), ("swiglu", True)):
        p = problem(T, 320, rows_for(T, 40), act=act, bias=True, residual=True, pad=pad, f32=f32, seed=7)
        check(p, call(m, p, pad_out=pad))


@pytest.mark.parametrize("T", [40, 300])
@pytest.mark.parametrize("more", [0, 1])
def test_residual_in_place(m, T, more):  # noqa: F811
    p = problem(T, 256, rows_for(T, more), residual=True, bias=True, seed=8)
    r = p["r"].cuda()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    check(p, m.linear_a16w4_mxfp4(p["x"].cuda(), torch.from_numpy(p["w"]).cuda(), torch.from_numpy(p["s"]).cuda(),
                                  bias=p["b"].cuda(), residual=r, out=r, workspace=ws))


@pytest.mark.parametrize("band", [(0, 1), (0, 40), (100, 150), (140, 175), (225, 240)])
def test_scale_bytes(m, band):  # noqa: F811
    p = problem(300, 256, rows_for(300), band=band, f32=True, seed=9)
    want, slack = linear.ref.linear(p["x"].double().numpy(), p["w"], p["s"])
    got = call(m, p).double().cpu().numpy()
    assert (np.abs(got - want) <= 257 * 2.0 ** -23 * slack + 256 * 2.0 ** -126).all()


@pytest.mark.parametrize("T", [40, 300])
def test_not_finite(m, T):  # noqa: F811
    p = problem(T, 256, rows_for(T), seed=10)
    p["s"][5, 3] = 255  # one block of weight row 5 is NaN
    p["x"][0, 7] = float("inf")  # column 7 is 0 in row 9, positive in row 11
    p["w"][9, 3] = 0
    p["w"][11, 3] = 0x20
    p["x"][T - 1, 9] = float("nan")
    got = call(m, p).float().cpu().numpy()
    assert np.isnan(got[:, 5]).all() and np.isnan(got[T - 1]).all()
    assert np.isnan(got[0, 9]) and got[0, 11] == np.inf
    got[:, 5] = 0
    assert np.isfinite(got[1: T - 1]).all()


def test_huge_activations(m):  # noqa: F811
    for T in (40, 300):
        p = problem(T, 64, rows_for(T), f32=True, seed=11)
        p["x"] = (p["x"].double() * 2.0 ** 112).bfloat16()
        check(p, call(m, p))


@pytest.mark.parametrize("T", [40, 100, 400])
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_repeatable(m, T, act):  # noqa: F811
    p = problem(T, 1024, rows_for(T, 300), act=act, bias=True, seed=13)
    first = call(m, p)
    for _ in range(3):
        assert torch.equal(call(m, p), first)


@pytest.mark.parametrize("T", [90, 400])
def test_captured(m, T):  # noqa: F811
    N = rows_for(T, 6)
    p = problem(T, 512, N, bias=True, residual=True, seed=14)
    x, w, s = on_gpu(p["x"]), torch.from_numpy(p["w"]).cuda(), torch.from_numpy(p["s"]).cuda()
    b, r = p["b"].cuda(), p["r"].cuda()
    out = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    m.linear_a16w4_mxfp4(x, w, s, bias=b, residual=r, out=out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.linear_a16w4_mxfp4(x, w, s, bias=b, residual=r, out=out, workspace=ws)
    q = problem(T, 512, N, bias=True, residual=True, seed=15)
    x.copy_(q["x"])
    r.copy_(q["r"])
    out.fill_(0)
    graph.replay()
    q.update(w=p["w"], s=p["s"], b=p["b"])
    check(q, out)


@pytest.mark.parametrize("act", [None, "gelu", "swiglu"])
@pytest.mark.parametrize("K", [64, 128, 192, 320, 352, 384, 416, 448, 480, 640, 1376, 1408, 1472, 1504, 2912, 4000])
def test_several_tiles_a_pair(m, K, act):  # noqa: F811
    """Steps that do not divide by four, by the stages or by the packed weights' stages, tile after tile."""
    both(m, 2500, K, 2600, act=act, bias=True, residual=True, seed=K)


@pytest.mark.parametrize("T,K,N", [(1208, 6080, 4096), (3020, 448, 1837), (4000, 1472, 2500), (300, 6080, 8192), (2100, 3584, 1500), (1208, 8192, 1024)])
def test_many_calls_agree(m, T, K, N):  # noqa: F811
    """Deep rows whose tiles of x come out of order: every call's result is the first's, and no wait runs out."""
    g = torch.Generator(device="cuda").manual_seed(K)
    xs = [torch.randn(T, K, generator=g, device="cuda").bfloat16() for _ in range(3)]
    w = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, generator=g, device="cuda")
    s = torch.randint(115, 122, (N, K // 32), dtype=torch.uint8, generator=g, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    flush = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")
    first = [m.linear_a16w4_mxfp4(x, w, s, workspace=ws) for x in xs]
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(240):
        if i % 8 == 0:
            flush.fill_(i)  # x comes from memory
        wrong += (m.linear_a16w4_mxfp4(xs[i % 3], w, s, workspace=ws) != first[i % 3]).sum()
    assert m.linear_read_status(ws) == 0 and wrong.item() == 0
