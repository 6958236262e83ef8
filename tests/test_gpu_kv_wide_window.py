"""Windows as wide as an int holds, and wider: with fewer keys than rows the first key of a window lies far below zero."""

import numpy as np
import pytest

from tests.test_gpu_kv_attention import both, check, m, problem, run  # noqa: F401  (m: the fixture)

pytestmark = pytest.mark.gpu

STREAMED = dict(lens=[40, 1, 30, 300, 0], qlens=[44, 9, 1, 7, 5], H=2, G=4, D=128, page=16)
PROMPTS = dict(lens=[40, 60, 200, 100], qlens=[44, 200, 203, 100], H=40, G=1, D=64, page=64)


@pytest.mark.parametrize("kind", [STREAMED, PROMPTS])
@pytest.mark.parametrize("window", [39, 2 ** 30, 2 ** 31 - 40, 2 ** 31 - 2, 2 ** 31 - 1])
def test_wide_windows(m, kind, window):  # noqa: F811
    both(m, problem(**kind, seed=5), scale=0.1, window=window)


@pytest.mark.parametrize("kind", [STREAMED, PROMPTS])
@pytest.mark.parametrize("window", [2 ** 31, 2 ** 32 + 3, 10 ** 12])
def test_windows_past_an_int_are_as_good_as_none(m, kind, window):  # noqa: F811
    p = problem(**kind, seed=6)
    out, lse = run(m, p, 0.1, window=window)
    check(p, out, lse, 0.1)


def test_window_beside_cut_rows(m):  # noqa: F811
    p = problem([300, 40], [60, 44], 2, 4, 128, 16, seed=7)
    out, lse = run(m, p, 0.1, window=2 ** 31 - 1, max_q=3)
    rows = np.concatenate([np.arange(3), 60 + np.arange(3)])
    full, full_lse = run(m, p, 0.1)
    assert (out[rows] - full[rows]).abs().max() < 2e-2 and np.array_equal((lse[rows] == -np.inf).cpu(), (full_lse[rows] == -np.inf).cpu())
