"""The linear layer where K is split over the pairs of a cluster (two, three and four), with every epilogue: whichever pair
finishes a chunk of tokens applies bias, activation and residual to it.  The sizes say that they are split: the library's
own choice is asked.  The same float64 oracle and derived bound as for smaller ones."""

import ctypes

import numpy as np
import pytest
import torch

from tests import test_gpu_block_giveup as giveup
from tests.test_gpu_linear import call, check, m, on_gpu, problem  # noqa: F401

pytestmark = pytest.mark.gpu


def splits(m, T, K, N, act=None):  # noqa: F811
    cols = N // 2 if act == "swiglu" else N
    d = m._native.LinearStruct(T, K, N, {None: 0, "silu": 1, "gelu": 2, "swiglu": 3}[act], 0, K, cols, cols)
    return m._native.load().linear_mxfp4_splits(ctypes.byref(d))


def split_problem(m, n, T, K, N, act=None, **kw):  # noqa: F811
    """A problem whose K is split in ``n``."""
    assert splits(m, T, K, N, act) == n, (T, K, N, act)
    return problem(T, K, N, act=act, **kw)


# pairs, rows, depth, weight rows: fewer chunks of 16 tokens than pairs, as many, a tile and a part of one; quads that do not
# divide by the pairs; the last quad a part
SIZES = [(2, 260, 1312, 1250), (2, 400, 2048, 800), (3, 40, 2080, 2500), (3, 150, 2336, 1250), (3, 300, 2752, 600),
         (4, 40, 2912, 2500), (4, 150, 3584, 1250), (4, 256, 8192, 700), (4, 300, 4128, 600)]


@pytest.mark.parametrize("n,T,K,N", SIZES)
@pytest.mark.parametrize("act", [None, "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("bias,residual,f32", [(False, False, False), (True, False, True), (False, True, True), (True, True, False)])
def test_epilogues(m, n, T, K, N, act, bias, residual, f32):  # noqa: F811
    p = split_problem(m, n, T, K, N, act, bias=bias, residual=residual, f32=f32, seed=1)
    check(p, call(m, p))


@pytest.mark.parametrize("n,T,K,N", SIZES)
@pytest.mark.parametrize("pad", [1, 8])
def test_strided_rows(m, n, T, K, N, pad):  # noqa: F811
    for act, f32 in ((None, False), ("swiglu", True)):
        p = split_problem(m, n, T, K, N, act, bias=True, residual=True, pad=pad, f32=f32, seed=2)
        check(p, call(m, p, pad_out=pad))


@pytest.mark.parametrize("n,T,K,N", SIZES)
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_residual_in_place(m, n, T, K, N, act):  # noqa: F811
    p = split_problem(m, n, T, K, N, act, bias=True, residual=True, seed=3)
    r = p["r"].cuda()
    check(p, m.linear_a16w4_mxfp4(p["x"].cuda(), torch.from_numpy(p["w"]).cuda(), torch.from_numpy(p["s"]).cuda(),
                                  bias=p["b"].cuda(), act=act, residual=r, out=r))


@pytest.mark.parametrize("n,T,K,N", SIZES)
def test_not_finite(m, n, T, K, N):  # noqa: F811
    p = split_problem(m, n, T, K, N, seed=4)
    p["s"][5, -1] = 255  # the last block of weight row 5 is NaN
    p["x"][0, 7] = float("inf")  # column 7 is 0 in row 9, positive in row 11
    p["w"][9, 3] = 0
    p["w"][11, 3] = 0x20
    p["x"][T - 1, K - 1] = float("nan")
    got = call(m, p).float().cpu().numpy()
    assert np.isnan(got[:, 5]).all() and np.isnan(got[T - 1]).all()
    assert np.isnan(got[0, 9]) and got[0, 11] == np.inf
    got[:, 5] = 0
    assert np.isfinite(got[1: T - 1]).all()


@pytest.mark.parametrize("n,T,K,N", SIZES)
def test_unlike_sizes(m, n, T, K, N):  # noqa: F811
    """Values and scale bytes of very unlike size, some pairs' runs of K far below the others'."""
    g = np.random.default_rng(K)
    p = split_problem(m, n, T, K, N, bias=True, f32=True, seed=5)
    x = p["x"].double().numpy().copy()
    for k in range(0, K, 256):
        x[:, k: k + 256] *= 2.0 ** g.integers(-40, 20)
    p["x"] = torch.from_numpy(x).bfloat16()
    p["s"][::3] = g.integers(60, 160, p["s"][::3].shape)
    p["s"][1::7] = 0
    check(p, call(m, p))


@pytest.mark.parametrize("n,T,K,N", SIZES)
@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_repeatable_and_captured(m, n, T, K, N, act):  # noqa: F811
    p = split_problem(m, n, T, K, N, act, bias=True, residual=True, seed=6)
    x, w, s = on_gpu(p["x"]), torch.from_numpy(p["w"]).cuda(), torch.from_numpy(p["s"]).cuda()
    b, r = p["b"].cuda(), p["r"].cuda()
    out, ws = torch.empty_like(r), torch.zeros(256, dtype=torch.uint8, device="cuda")

    def run():
        m.linear_a16w4_mxfp4(x, w, s, bias=b, act=act, residual=r, out=out, workspace=ws)

    run()
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        out.fill_(0)
        graph.replay()
        assert torch.equal(out, first)
    q = problem(T, K, p["N"], act=act, bias=True, residual=True, seed=7)
    x.copy_(q["x"])
    r.copy_(q["r"])
    graph.replay()
    q.update(w=p["w"], s=p["s"], b=p["b"])
    check(q, out)
    assert m.linear_read_status(ws) == 0


@pytest.mark.parametrize("n,T,K,N,act", [(2, 400, 2048, 800, "silu"), (3, 150, 2336, 1250, "gelu"), (4, 40, 2912, 2500, "swiglu")])
def test_waits_that_run_out(m, n, T, K, N, act):  # noqa: F811
    assert splits(m, T, K, N, act) == n
    giveup.check_linear(m, T, K, N, act)


def test_the_choice(m):  # noqa: F811
    assert splits(m, 1, 3584, 4608) == 0 and splits(m, 32, 65536, 4096) == 0  # few rows: from registers
    assert splits(m, 0, 64, 64) == 0
    assert splits(m, 2048, 256, 4096) == 1  # many tiles
    assert splits(m, 10, 48, 64) == -2 and m._native.load().linear_mxfp4_splits(None) == -1
