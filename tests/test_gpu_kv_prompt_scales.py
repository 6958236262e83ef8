"""The tensor-core kernel's f16 product over the whole range of scale bytes that it takes (104 .. 140, and 0), in requests
whose rows see more than 256 keys.  The bound of test_gpu_kv_attention.py, and half of the f16 weights' step, 2^-24 in units
of 2^-9, of the sum of the visible |v|."""

import numpy as np
import pytest

from oracle import kv_cache as ref
from tests.test_gpu_kv_attention import m, problem, run  # noqa: F401  (m: the fixture)

pytestmark = pytest.mark.gpu

H = 40


@pytest.mark.parametrize("G,D", [(1, 64), (1, 128), (3, 128)])
@pytest.mark.parametrize("keys,values,scale", [
    ((104, 112), (104, 112), 50.0), ((104, 140), (104, 140), 2e-5), ((138, 140), (138, 140), 1e-5), ((113, 113), (112, 113), 3.0),
    ((0, 0), (104, 105), 1.0), ((120, 127), (0, 0), 0.2), ((126, 127), (104, 140), 0.3),
])
def test_scale_bytes_of_the_range(m, G, D, keys, values, scale):  # noqa: F811
    # a chunk of a long prompt, a prompt's end, a single token beside them; the last request is short
    p = problem([700, 400, 513, 120], [90, 120, 1, 120], H, G, D, 64, seed=D + G, bands=(keys, values))
    out, lse = run(m, p, scale)
    kv = [0, 21, H - 1]
    hq = [h * G + i for h in kv for i in range(G)]
    want, wl, spread, size = ref.attention(p["q"].float().numpy()[:, hq], p["data"][:, kv], p["table"], p["lens"], p["start"], scale)
    got, gl = out.double().cpu().numpy()[:, hq], lse.double().cpu().numpy()[:, hq]
    err = D * 2.0 ** -24 * size
    bound = (2.0 ** -9 + 2.0 ** -13) * np.abs(want) + (2.0 ** -9 + 2.0 ** -13 + 2 * err[..., None]) * spread + 1e-37
    for r, n in enumerate(p["lens"]):  # (all keys, also those past a row's position)
        _, _, vc, vs = ref.read(p["data"][:, kv], p["table"][r, np.arange(n) // 64] * 64 + np.arange(n) % 64)
        total = np.abs(ref.values(vc, vs)).sum(0)  # [heads, D]
        bound[p["start"][r]: p["start"][r + 1]] += 2.0 ** -34 * np.repeat(total, G, 0)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (bad.mean(), np.argwhere(bad)[:3], got[bad][:4], want[bad][:4], bound[bad][:4])
    off = ~(np.abs(gl - wl) <= err + 2.0 ** -20 * (1 + np.abs(wl)))
    assert not off.any(), (gl[off][:4], wl[off][:4])
