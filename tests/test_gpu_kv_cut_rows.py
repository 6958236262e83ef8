"""Requests with more rows than max_q_len, or past the rows of q: the rows that are written sit at the positions that the
request's true row count gives them, the others stay as they were."""

import numpy as np
import pytest
import torch

from oracle import kv_cache as ref
from tests.test_gpu_kv_attention import m, problem, run  # noqa: F401  (m: the fixture)

pytestmark = pytest.mark.gpu


def compare(p, out, lse, rows, causal, window, scale=0.1):
    """``rows``: the rows of q that are to be written.  The bound of test_gpu_kv_attention.py; requests of the
    tensor-core kernel whose rows see more than 256 keys: plus 2^-34 of the values' sum (at most 6 x 1,024)."""
    want, wl, spread, size = ref.attention(p["q"].float().numpy(), p["data"], p["table"], p["lens"], p["start"], scale,
                                           causal, window)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    left = np.setdiff1d(np.arange(len(got)), rows)
    assert (got[left] == 77.0).all() and (gl[left] == 77.0).all()
    got, gl, want, wl, spread, size = (x[rows] for x in (got, gl, want, wl, spread, size))
    D = p["D"]
    bound = ((2.0 ** -9 + 2.0 ** -13) * np.abs(want) +
             (2.0 ** -9 + 2.0 ** -13 + 2 * D * 2.0 ** -24 * size[..., None]) * spread + 2.0 ** -34 * 6 * 1024)
    assert (np.abs(got - want) <= bound).all()
    seen = np.isfinite(wl)
    assert np.array_equal(gl[~seen], wl[~seen])
    gl, wl, size = gl[seen], wl[seen], size[seen]
    assert (np.abs(gl - wl) <= D * 2.0 ** -24 * size + 2.0 ** -20 * (1 + np.abs(wl))).all()


STREAMED = dict(lens=[300, 50, 7, 40, 1], qlens=[9, 4, 9, 40, 3], H=2, G=4, D=128, page=16)
PROMPTS = dict(lens=[700, 257, 60, 513], qlens=[200, 257, 200, 33], H=40, G=1, D=64, page=64)


@pytest.mark.parametrize("kind,most", [(STREAMED, 1), (STREAMED, 4), (STREAMED, 8), (PROMPTS, 40), (PROMPTS, 150)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 5), (True, 200), (False, 0)])
def test_longer_requests_than_max_q_len(m, kind, most, causal, window):  # noqa: F811
    p = problem(**kind, seed=most)
    out, lse = run(m, p, 0.1, causal=causal, window=window, max_q=most)
    rows = np.concatenate([np.arange(a, min(b, a + most)) for a, b in zip(p["start"], p["start"][1:])])
    compare(p, out, lse, rows, causal, window)


@pytest.mark.parametrize("kind,cut", [(STREAMED, 2), (STREAMED, 20), (PROMPTS, 3), (PROMPTS, 133)])
@pytest.mark.parametrize("window", [0, 30])
def test_requests_past_the_rows_of_q(m, kind, cut, window):  # noqa: F811
    p = problem(**kind, seed=cut)
    q = p["q"].cuda()[:-cut].contiguous()
    out, lse = run(m, p, 0.1, window=window, q=q)
    compare(p, out, lse, np.arange(len(q)), True, window)
