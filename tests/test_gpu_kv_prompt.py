"""The tensor-core kernel of the attention over the 4-bit cache, at requests x heads that fill the GPU (with fewer,
requests of this size are streamed): the float64 oracle and the bound of test_gpu_kv_attention.py.

Where rows see more than 256 keys, weights have 11 bits, those below 2^-23 of the largest a multiple of 2^-34 of it
(2^-25 in f16 at 2^9): the bound there also has 2^-34 of sum |v| over the visible keys.
"""

import numpy as np
import pytest
import torch

from oracle import kv_cache as ref
from tests.test_gpu_kv_attention import both, check, m, problem, run  # noqa: F401  (m: the fixture)

pytestmark = pytest.mark.gpu

# 4 requests x 40 kv heads: one for every SM, rows above 32 go to the tensor cores
H = 40


def long_check(p, out, lse, scale, causal=True, window=0):
    want, wl, spread, size = ref.attention(p["q"].float().numpy(), p["data"], p["table"], p["lens"], p["start"], scale,
                                           causal, window)
    D = p["D"]
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    # the largest value of the bands used here is 6, at most 1,024 keys
    bound = ((2.0 ** -9 + 2.0 ** -13) * np.abs(want) +
             (2.0 ** -9 + 2.0 ** -13 + 2 * D * 2.0 ** -24 * size[..., None]) * spread + 2.0 ** -34 * 6 * 1024)
    assert (np.abs(got - want) <= bound).all()
    seen = np.isfinite(wl)
    assert np.array_equal(gl[~seen], wl[~seen])
    gl, wl, size = gl[seen], wl[seen], size[seen]
    assert (np.abs(gl - wl) <= D * 2.0 ** -24 * size + 2.0 ** -20 * (1 + np.abs(wl))).all()


@pytest.mark.parametrize("G,D,page", [(1, 128, 64), (2, 64, 16), (3, 128, 256)])
@pytest.mark.parametrize("window", [0, 30, 300])
def test_prompts(m, G, D, page, window):  # noqa: F811
    # ragged lengths; a request whose first rows see nothing, one of a single token beside the prompts
    p = problem([700, 257, 40, 513], [90, 257, 44, 1], H, G, D, page, seed=G)
    out, lse = run(m, p, 0.2, window=window)
    long_check(p, out, lse, 0.2, window=window)


@pytest.mark.parametrize("G,D", [(1, 64), (2, 128)])
@pytest.mark.parametrize("lens", [[64, 33, 256, 129], [1, 255, 128, 127]])
@pytest.mark.parametrize("scale", [0.1, 4.0, -30.0])
def test_few_keys_with_weights_of_any_size(m, G, D, lens, scale):  # noqa: F811
    # the bound without the extra term: 16-bit weights at any size
    both(m, problem(lens, [max(40, n // 2) for n in lens], H, G, D, 32, seed=lens[0]), scale=scale)


@pytest.mark.parametrize("window", [1, 17, 256])
def test_short_windows(m, window):  # noqa: F811
    both(m, problem([600, 300, 64, 90], [80, 45, 64, 33], H, 2, 128, 64, seed=window), scale=3.0, window=window)


@pytest.mark.parametrize("bands,n", [(((96, 110), (120, 127)), 100), (((96, 110), (120, 127)), 400),
                                     (((120, 127), (30, 200)), 100), (((120, 127), (30, 200)), 400),
                                     (((104, 140), (104, 113)), 100), (((254, 255), (0, 0)), 100)])
def test_scale_bytes_outside_the_kernels_range(m, bands, n):  # noqa: F811
    # requests 1 and 3 keep usual scales: only the others are marked and done again
    p = problem([n, n], [50, 60], H, 1, 64, 64, bands=bands, seed=n)
    usual = problem([n, n], [50, 60], H, 1, 64, 64, seed=n + 1)
    p["data"] = np.concatenate([p["data"], usual["data"]])
    usual_table = np.where(usual["table"] >= 0, usual["table"] + p["pages"], usual["table"])
    p["table"] = np.concatenate([p["table"], usual_table])
    p["pages"] += usual["pages"]
    p["lens"] = np.concatenate([p["lens"], usual["lens"]])
    p["start"] = np.concatenate([p["start"], usual["start"][1:] + p["start"][-1]])
    p["q"] = torch.cat([p["q"], usual["q"]])
    # scores of usual scales small enough that no weight falls below the 11 bits' range
    both(m, p, scale=0.01)


def test_every_key_is_seen_without_the_mask(m):  # noqa: F811
    p = problem([300, 128, 77, 640], [40, 50, 33, 64], H, 2, 64, 16, seed=9)
    out, lse = run(m, p, 0.2, causal=False)
    long_check(p, out, lse, 0.2, causal=False)


def test_equal_scores(m):  # noqa: F811
    # all weights 1: the largest sums
    p = problem([640, 256, 129, 1024], [40, 70, 64, 36], H, 1, 128, 64, seed=4)
    p["q"].zero_()
    both(m, p, scale=0.3)
