"""GPU parity of the linear layer on MXFP4 weights with the float64 oracle.

Bound per result, from the arithmetic alone.  Weights and activations enter
exactly, so h is a float32 sum of K products and the bias: whatever the order,
off by at most (K + 1) 2^-23 of size = sum |x w| + |b| (2^-24 an addition where it
rounds to nearest, 2^-23 where the matrix unit cuts off).  The activation passes that on
times its slope (the oracle's ``slack``) and adds a few units in the last place of
its own exponential, quotient and product, which 2^-18 of the result and of
``slack`` covers (the exponential's argument is below 2^7 where it matters, 2^7
2^-25).  The residual's sum and the result round once each: 2^-24, and 2^-8 for bf16.
    |out - ref| <= ((K + 1) 2^-23 + 2^-18 [act]) slack + (2^-18 [act] + 2^-23 + 2^-8 [bf16]) |ref| + 2^-23 |residual|
"""

import numpy as np
import pytest
import torch

from oracle import block as ref
from oracle import formats

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mxfp4_weight_only_gb300 import build

    build.build()
    import mxfp4_weight_only_gb300 as m

    return m


def problem(T, K, N, act=None, bias=False, residual=False, f32=False, seed=0, band=(119, 123), pad=0):
    g = np.random.default_rng(seed + 7 * T + K + N)
    cols = N // 2 if act == "swiglu" else N
    bf = lambda *s: torch.from_numpy(g.standard_normal(s)).to(torch.bfloat16)  # noqa: E731
    p = dict(T=T, K=K, N=N, cols=cols, act=act, f32=f32)
    p["x"] = bf(T, K + 8 * pad)[:, 8 * pad // 2 // 8 * 8:][:, :K]
    p["w"] = g.integers(0, 256, (N, K // 2), dtype=np.uint8)
    p["s"] = g.integers(band[0], band[1] + 1, (N, K // 32), dtype=np.uint8)
    p["b"] = bf(N) if bias else None
    p["r"] = bf(T, cols + pad)[:, :cols] if residual else None
    return p


def on_gpu(t):
    """The tensor on the GPU with its strides."""
    if t is None:
        return None
    wide = torch.full((t.shape[0], t.stride(0)), 1e30, dtype=t.dtype, device="cuda")
    wide[:, : t.shape[1]] = t
    return wide[:, : t.shape[1]]


def call(m, p, pad_out=0, **kw):
    dt = torch.float32 if p["f32"] else torch.bfloat16
    wide = torch.full((p["T"], p["cols"] + pad_out), 77.0, dtype=dt, device="cuda")
    out = wide[:, : p["cols"]]
    ws = torch.zeros(max(256, m.linear_workspace_bytes(p["T"], p["N"], p["K"])), dtype=torch.uint8, device="cuda")
    got = m.linear_a16w4_mxfp4(on_gpu(p["x"]), torch.from_numpy(p["w"]).cuda(), torch.from_numpy(p["s"]).cuda(),
                               bias=None if p["b"] is None else p["b"].cuda(), act=p["act"], residual=on_gpu(p["r"]),
                               out=out, workspace=ws, **kw)
    assert got is out
    assert m.linear_read_status(ws) == 0
    assert (wide[:, p["cols"]:] == 77.0).all()
    return out


def check(p, out):
    num = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    want, slack = ref.linear(num(p["x"]), p["w"], p["s"], num(p["b"]), p["act"], num(p["r"]))
    got = out.double().cpu().numpy()
    a = 2.0 ** -18 if p["act"] else 0.0
    bound = ((p["K"] + 1) * 2.0 ** -23 + a) * slack + (a + 2.0 ** -23 + (0 if p["f32"] else 2.0 ** -8)) * np.abs(want)
    if p["r"] is not None:
        bound = bound + 2.0 ** -23 * np.abs(num(p["r"]))
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], bound[bad][:4])


def both(m, *a, **kw):
    p = problem(*a, **kw)
    check(p, call(m, p))


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 200, 255, 256, 257, 300, 513])
def test_rows(m, T):
    both(m, T, 256, 160, seed=1)


@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 480, 992, 1024, 2080, 4096, 8192])
@pytest.mark.parametrize("T", [1, 5, 40, 150, 300])
def test_depths(m, K, T):
    both(m, T, K, 72, seed=2, bias=True)


@pytest.mark.parametrize("N", [1, 2, 3, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 255, 256, 257, 500, 1111])
@pytest.mark.parametrize("T", [1, 13, 70, 260])
def test_columns(m, N, T):
    both(m, T, 192, N, seed=3, bias=True, residual=True)


@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("T,N", [(17, 2), (18, 34), (24, 1110), (25, 62), (32, 5000)])
@pytest.mark.parametrize("K", [32, 96, 1056, 3200, 8224])  # a part of a chunk .. more chunks than a warp has on the way
def test_up_to_32_rows(m, T, N, K, act):
    both(m, T, K, N, act=act, bias=True, residual=True, seed=22)


@pytest.mark.parametrize("T", [1, 33, 300])
def test_small_gated_and_deepest(m, T):
    for N in (2, 4, 30, 34, 258):
        both(m, T, 96, N, act="swiglu", bias=True, residual=True, seed=19)
    both(m, T, 65536, 5, bias=True, seed=20)


@pytest.mark.parametrize("T", [2, 50, 300])
@pytest.mark.parametrize("K", [32, 96, 160, 2080])
@pytest.mark.parametrize("skip", [1, 2, 3])
def test_scales_at_any_address(m, T, K, skip):
    """Scale rows of an odd length that begin anywhere: slices of a taller array, whose other rows are NaN."""
    p = problem(T, K, 50, seed=21)
    tall = torch.full((50 + 2 * skip, K // 32), 255, dtype=torch.uint8, device="cuda")
    s = tall[skip: skip + 50]
    s.copy_(torch.from_numpy(p["s"]))
    check(p, m.linear_a16w4_mxfp4(on_gpu(p["x"]), torch.from_numpy(p["w"]).cuda(), s))


@pytest.mark.parametrize("act", [None, "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("bias,residual,f32", [(False, False, False), (True, False, True), (False, True, True), (True, True, False)])
@pytest.mark.parametrize("T", [3, 50, 140, 600])
def test_epilogues(m, act, bias, residual, f32, T):
    both(m, T, 288, 154, act=act, bias=bias, residual=residual, f32=f32, seed=4)
    both(m, T, 512, 256, act=act, bias=bias, residual=residual, f32=f32, seed=5)


@pytest.mark.parametrize("T", [1, 20, 130, 520])
@pytest.mark.parametrize("pad", [1, 3, 8])
def test_strided_rows(m, T, pad):
    p = problem(T, 320, 144, bias=True, residual=True, pad=pad, seed=6)
    check(p, call(m, p, pad_out=pad))
    p = problem(T, 320, 144, act="swiglu", residual=True, pad=pad, f32=True, seed=6)
    check(p, call(m, p, pad_out=pad))


@pytest.mark.parametrize("T", [1, 8, 40, 300])
@pytest.mark.parametrize("N", [96, 97])
def test_residual_in_place(m, T, N):
    p = problem(T, 256, N, residual=True, bias=True, seed=8)
    r = p["r"].cuda()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    got = m.linear_a16w4_mxfp4(p["x"].cuda(), torch.from_numpy(p["w"]).cuda(), torch.from_numpy(p["s"]).cuda(),
                               bias=p["b"].cuda(), residual=r, out=r, workspace=ws)
    check(p, got)


@pytest.mark.parametrize("T", [1, 30, 300])
@pytest.mark.parametrize("band", [(0, 1), (0, 40), (100, 150), (140, 175), (225, 240)])
def test_scale_bytes(m, T, band):
    # results of any size a float32 holds; the small ones to the smallest normal float32
    p = problem(T, 256, 80, band=band, f32=True, seed=9)
    num = p["x"].double().numpy()
    want, slack = ref.linear(num, p["w"], p["s"])
    got = call(m, p).double().cpu().numpy()
    assert (np.abs(got - want) <= 257 * 2.0 ** -23 * slack + 256 * 2.0 ** -126).all()


@pytest.mark.parametrize("T", [1, 30, 300])
def test_not_finite(m, T):
    p = problem(T, 256, 80, seed=10)
    p["s"][5, 3] = 255  # one block of weight row 5 is NaN
    p["x"][0, 7] = float("inf")  # column 7 is 0 in row 9, positive in row 11
    p["w"][9, 3] = 0
    p["w"][11, 3] = 0x20
    if T > 1:
        p["x"][T - 1, 9] = float("nan")
    got = call(m, p).float().cpu().numpy()
    assert np.isnan(got[:, 5]).all()
    assert np.isnan(got[0, 9]) and got[0, 11] == np.inf
    if T > 1:
        assert np.isnan(got[T - 1]).all()
        fine = np.ones((T, 80), bool)
        fine[[0, T - 1]] = False
        fine[:, 5] = False
        assert np.isfinite(got[fine]).all()


@pytest.mark.parametrize("T", [1, 3, 8, 9, 16, 20, 40])
@pytest.mark.parametrize("K", [96, 128, 1056, 4096])
def test_unlike_sizes(m, T, K):
    """Values and scale bytes of very unlike size side by side, in some chunks of K only: what a kernel may hold in
    fewer exponent bits has to be noticed."""
    g = np.random.default_rng(T + K)
    p = problem(T, K, 70, f32=True, seed=17)
    x = p["x"].double().numpy().copy()
    for k in range(0, K, 64):
        kind = (k // 64) % 6
        part = x[:, k: k + 32]
        if kind == 0:
            part *= 2.0 ** g.integers(-60, 1, part.shape)  # values far below the largest
        elif kind == 1:
            part[:] = 0.0
        elif kind == 2:
            part *= 2.0 ** -115  # close to the smallest normal number
        elif kind == 3:
            part *= 2.0 ** g.integers(-20, 20, (T, 1))  # tokens of unlike size
        elif kind == 4:
            part[:, ::2] = 0.0
            part[:, 1::2] *= 2.0 ** -40
    p["x"] = torch.from_numpy(x).bfloat16()
    s = p["s"]
    s[::3, ::2] = g.integers(60, 160, s[::3, ::2].shape)  # scales far apart in a row
    s[1::7] = 0  # rows of the smallest scale
    s[2::9, 0] = 0
    p["w"][2::9, :16] = 0  # a block of zeros, as the conversion writes it
    check(p, call(m, p))


@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("T", [1, 3, 8, 9, 16])
@pytest.mark.parametrize("K,N", [(32, 4866), (96, 12002), (1056, 7300), (2048, 7298), (3200, 9800), (8192, 5000)])
def test_tiles_walked(m, T, K, N, act):
    """More tiles of 16 rows than two an SM: a last round that is not full, tiles past the end, parts of chunks."""
    both(m, T, K, N, act=act, bias=True, residual=True, f32=T == 3, seed=23)


@pytest.mark.parametrize("T", [1, 9])
def test_tiles_walked_not_finite(m, T):
    p = problem(T, 1056, 6000, seed=24)
    p["s"][5999, 32] = 255  # the last block of the last row is NaN
    p["x"][T - 1, 1055] = float("inf")  # 0 in row 17, positive in row 18
    p["w"][17, -1] = 0
    p["w"][18, -1] = 0x20
    got = call(m, p).float().cpu().numpy()
    assert np.isnan(got[:, 5999]).all() and np.isnan(got[T - 1, 17]) and got[T - 1, 18] == np.inf
    assert np.isfinite(got[: T - 1, :5999]).all()


@pytest.mark.parametrize("T", [1, 7, 16])
@pytest.mark.parametrize("K,N", [(128, 20000), (4096, 5500), (32768, 33), (8192, 700), (32, 16)])
def test_many_tiles_and_deep_rows(m, T, K, N):
    p = problem(T, K, N, bias=True, residual=True, seed=18)
    check(p, call(m, p))


def test_gelu_of_every_size(m):
    """h itself by a weight of ones on the diagonal, against h Phi(h).  The kernel's max(h, 0) - |h| q, q = Phi(-|h|) as
    t P(t) e^(-h^2/2): the fit of P 2^-24.8 of it, t off by 2^-22 at a sensitivity of at most 2.4, eight steps of P 2^-22.4,
    the exponential 2^-22 and two roundings of its argument, h^2 2^-24, two products 2^-23: below (2^-19 + h^2 2^-24) |h| q."""
    special = pytest.importorskip("scipy.special")
    h = torch.cat([torch.linspace(-14, 14, 4000), torch.randn(4000), torch.randn(4000) * 0.01, torch.tensor(
        [0.0, -0.0, 8.0, -8.0, 8.0625, 30.0, -30.0, 1e30, -1e30, float("inf"), float("nan")] + [0.0] * 21)]).bfloat16()
    h = h[: h.numel() // 32 * 32].reshape(-1, 32)
    w = np.zeros((32, 16), np.uint8)
    for k in range(32):
        w[k, k // 2] = 0x20 if k % 2 else 0x02
    s = torch.full((32, 1), 127, dtype=torch.uint8, device="cuda")
    h[~torch.isfinite(h)] = 0  # (an infinity would meet the weight's zeros)
    for T in (1, 9, 20, h.shape[0]):
        x = h[-T:].cuda()
        out = m.linear_a16w4_mxfp4(x, torch.from_numpy(w).cuda(), s, act="gelu", out_dtype=torch.float32).double().cpu().numpy()
        v = h[-T:].double().numpy()
        want, q = v * special.ndtr(v), special.ndtr(-np.abs(v))
        assert (np.abs(out - want) <= (2.0 ** -19 + v * v * 2.0 ** -24) * np.abs(v) * q + 2.0 ** -24 * np.abs(want) + 1e-37).all()


def test_huge_activations(m):
    # products of 2^120, sums within float32
    for T in (1, 40, 300):
        p = problem(T, 64, 48, f32=True, seed=11)
        p["x"] = (p["x"].double() * 2.0 ** 112).bfloat16()
        check(p, call(m, p))


def test_other_stream_and_device_order(m):
    p = problem(200, 512, 320, act="gelu", bias=True, seed=12)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = [on_gpu(p["x"]), torch.from_numpy(p["w"]).cuda(), torch.from_numpy(p["s"]).cuda()]
    b = p["b"].cuda()
    torch.cuda.synchronize()
    out = m.linear_a16w4_mxfp4(*a, bias=b, act="gelu", stream=s)
    s.synchronize()
    check(p, out)


@pytest.mark.parametrize("T", [1, 24, 100, 400])
def test_repeatable(m, T):
    p = problem(T, 1024, 272, act="swiglu", bias=True, seed=13)
    first = call(m, p)
    for _ in range(3):
        assert torch.equal(call(m, p), first)


@pytest.mark.parametrize("T", [1, 20, 90, 400])
def test_captured(m, T):
    p = problem(T, 512, 208, bias=True, residual=True, seed=14)
    x, w, s = on_gpu(p["x"]), torch.from_numpy(p["w"]).cuda(), torch.from_numpy(p["s"]).cuda()
    b, r = p["b"].cuda(), p["r"].cuda()
    out = torch.empty(T, 208, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    m.linear_a16w4_mxfp4(x, w, s, bias=b, residual=r, out=out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.linear_a16w4_mxfp4(x, w, s, bias=b, residual=r, out=out, workspace=ws)
    q = problem(T, 512, 208, bias=True, residual=True, seed=15)
    x.copy_(q["x"])
    r.copy_(q["r"])
    out.fill_(0)
    graph.replay()
    q.update(w=p["w"], s=p["s"], b=p["b"])
    check(q, out)


def test_refusals(m):
    p = problem(4, 64, 32, seed=16)
    x, w, s = p["x"].cuda(), torch.from_numpy(p["w"]).cuda(), torch.from_numpy(p["s"]).cuda()
    for kw, e in ((dict(act="relu6"), ValueError), (dict(bias=torch.zeros(31, dtype=torch.bfloat16, device="cuda")), ValueError),
                  (dict(bias=torch.zeros(32, device="cuda")), TypeError), (dict(out_dtype=torch.float16), TypeError),
                  (dict(residual=torch.zeros(4, 33, dtype=torch.bfloat16, device="cuda")), ValueError),
                  (dict(workspace=torch.zeros(128, dtype=torch.uint8, device="cuda")), m.MoeError),
                  (dict(out=x[:, :32]), m.MoeError)):
        with pytest.raises(e):
            m.linear_a16w4_mxfp4(x, w, s, **kw)
    with pytest.raises(ValueError):
        m.linear_a16w4_mxfp4(x, w[:31], s[:31], act="swiglu")
    with pytest.raises(ValueError):
        m.linear_a16w4_mxfp4(x.t(), w, s)
    with pytest.raises(m.MoeError):  # rows 8 bytes apart from alignment
        wide = torch.zeros(4, 68, dtype=torch.bfloat16, device="cuda")
        m.linear_a16w4_mxfp4(wide[:, :64], w, s)
    assert m.linear_a16w4_mxfp4(x[:0], w, s).shape == (0, 32)
    torch.cuda.synchronize()


def test_matches_the_dequantised_weight(m):
    """The values are those of the MoE's weights: the same decoding."""
    g = np.random.default_rng(3)
    w, s = formats.quantize_mxfp4(g.standard_normal((48, 96)))
    x = torch.eye(96, dtype=torch.bfloat16)
    out = m.linear_a16w4_mxfp4(x.cuda(), torch.from_numpy(w).cuda(), torch.from_numpy(s).cuda(), out_dtype=torch.float32)
    assert np.array_equal(out.double().cpu().numpy(), formats.dequant_mxfp4(w, s).T)
