"""The first rows of a long prompt see few keys: their weights have 16 bits at any size, as those of a short prompt."""

import numpy as np
import pytest
import torch

from oracle import kv_cache as ref
from tests.test_gpu_kv_attention import m, problem, run  # noqa: F401  (m: the fixture)

pytestmark = pytest.mark.gpu

H = 40  # with four requests, one for every SM: rows above 32 go to the tensor cores


def compare(p, out, lse, scale, window=0):
    """The bound of test_gpu_kv_attention.py where a row sees at most 256 positions; else plus 2^-34 of the values' sum
    (weights of 11 bits: half of f16's step 2^-24 in units of 2^-9; values up to 6, at most 1,024)."""
    kv = [0, 18, H - 1]  # the heads looked at: the oracle is slow
    hq = [h * p["G"] + i for h in kv for i in range(p["G"])]
    want, wl, spread, size = ref.attention(p["q"].float().numpy()[:, hq], p["data"][:, kv], p["table"], p["lens"], p["start"],
                                           scale, True, window)
    D = p["D"]
    got, gl = out.double().cpu().numpy()[:, hq], lse.double().cpu().numpy()[:, hq]
    bound = (2.0 ** -9 + 2.0 ** -13) * np.abs(want) + (2.0 ** -9 + 2.0 ** -13 + 2 * D * 2.0 ** -24 * size[..., None]) * spread
    for r, n in enumerate(p["lens"]):
        a, b = p["start"][r], p["start"][r + 1]
        seen = n - (b - a) + np.arange(b - a) + 1
        if window:
            seen = np.minimum(seen, window)
        bound[a:b][seen > 256] += 2.0 ** -34 * 6 * 1024
    bad = np.abs(got - want) > bound + 1e-37
    assert not bad.any(), (np.unique(np.argwhere(bad)[:, 0]), got[bad][:4], want[bad][:4], bound[bad][:4])
    seen = np.isfinite(wl)
    assert np.array_equal(gl[~seen], wl[~seen])
    gl, wl, size = gl[seen], wl[seen], size[seen]
    assert (np.abs(gl - wl) <= D * 2.0 ** -24 * size + 2.0 ** -20 * (1 + np.abs(wl))).all()


@pytest.mark.parametrize("G,D", [(1, 64), (2, 128), (3, 64)])
@pytest.mark.parametrize("scale", [4.0, -30.0])
def test_sharp_weights(m, G, D, scale):  # noqa: F811
    # whole prompts; a chunk that begins at key 200; rows before the first key
    p = problem([600, 290, 700, 300], [600, 290, 500, 330], H, G, D, 64, seed=G)
    out, lse = run(m, p, scale)
    compare(p, out, lse, scale)


@pytest.mark.parametrize("G,D", [(1, 128), (5, 64)])
@pytest.mark.parametrize("window", [0, 257, 400])
def test_values_under_light_weights(m, G, D, window):  # noqa: F811
    """One key has nearly all the weight and no value; what is left weighs 2^-111 of it."""
    p = problem([520, 300, 410, 300], [520, 300, 300, 300], H, G, D, 32, seed=4)
    p["q"] = torch.ones_like(p["q"])
    NB = D // 32
    for r in range(4):
        for j in range(p["lens"][r]):
            rec = p["data"][p["table"][r, j // 32], :, j % 32 // 16]
            heavy = j % 150 == 3
            for b in range(D // 2):
                rec[:, ref.k_at(j % 16, b, D)] = 0x77 if heavy else 0xFF
                rec[:, ref.v_at(j % 16, b, D)] = 0x00 if heavy else 0x52 + j % 3
            rec[:, 16 * D + j % 16 * NB: 16 * D + (j % 16 + 1) * NB] = 127
            rec[:, 16 * D + D // 2 + j % 16 * NB: 16 * D + D // 2 + (j % 16 + 1) * NB] = 120
    scale = 0.05 * 128 / D
    out, lse = run(m, p, scale, window=window)
    compare(p, out, lse, scale, window)
