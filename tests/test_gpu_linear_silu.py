"""SiLU and SwiGLU of float32 results, as exact as float32 arithmetic is.

h itself by a weight of ones on the diagonal (so h is exact), against h / (1 + e^-h) in float64.  With e = exp(-|h|), off by two
units in the last place (2^-22; |h| is exact, so its size does not matter), 1 + e and h e round once each (2^-24) and the
quotient by two units (2^-22): below 2^-20 of the result.  SwiGLU multiplies once more, 2^-24.  Where e or the result is no
normal number (h below -83), 1e-37 on top."""

import numpy as np
import pytest
import torch

from tests.test_gpu_linear import m  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def diagonal(rows):
    """Weight [rows, rows] of ones on the diagonal: packed codes and scale bytes."""
    k = np.arange(rows)
    w = np.zeros((rows, rows // 2), np.uint8)
    w[k, k // 2] = np.where(k % 2, 0x20, 0x02)
    return w, np.full((rows, rows // 32), 127, np.uint8)


def values(T, K):
    g = np.random.default_rng(T)
    h = np.concatenate([np.linspace(-95, 95, 4000), g.standard_normal(4000) * 10, g.standard_normal(2000) * 0.01,
                        [0.0, -0.0, 30.0, -30.0, -86.0, -87.5, -88.5, -89.0, -100.0, 1e30, -1e30]])
    return torch.from_numpy(g.choice(h, (T, K))).bfloat16()


# streamed, walked (more than two tiles of 16 rows an SM), 17 and more rows, tensor cores
@pytest.mark.parametrize("T,K,copies", [(1, 64, 1), (9, 64, 1), (5, 64, 96), (24, 64, 1), (40, 96, 4), (300, 64, 64), (1000, 96, 9)])
@pytest.mark.parametrize("act", ["silu", "swiglu"])
def test_as_exact_as_float32(m, T, K, copies, act):  # noqa: F811
    w, s = (np.tile(a, (copies, 1)) for a in diagonal(K))
    if act == "swiglu":
        w, s = np.concatenate([w, w]), np.concatenate([s, s])
    x = values(T, K)
    out = m.linear_a16w4_mxfp4(x.cuda(), torch.from_numpy(w).cuda(), torch.from_numpy(s).cuda(), act=act, out_dtype=torch.float32)
    h = np.tile(x.double().numpy(), (1, copies))
    e = np.exp(-np.abs(h))
    want = np.where(h > 0, h, h * e) / (1 + e) * (h if act == "swiglu" else 1.0)
    with np.errstate(over="ignore", invalid="ignore"):
        want32 = np.where(np.abs(want) > 3.4e38, np.sign(want) * np.inf, want)
        off = ~(np.abs(out.double().cpu().numpy() - want32) <= (2.0 ** -20 + 2.0 ** -24) * np.abs(want) + 1e-37 * np.maximum(1, np.abs(h)))
        off &= ~(out.double().cpu().numpy() == want32)
    assert not off.any(), (off.sum(), h[off][:4], out.cpu().numpy()[off][:4], want[off][:4])
