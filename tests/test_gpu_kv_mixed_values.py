"""Values of all sizes in one request: a block of small values keeps them beside a block of huge ones, and a dimension's small
value beside a huge one that is zero there."""

import pytest

from tests.test_gpu_kv_attention import both, m, problem  # noqa: F401  (m: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,G,D", [(2, 4, 128), (3, 2, 64), (1, 16, 128)])
@pytest.mark.parametrize("bands", [(0, 250), (30, 250), (200, 250), (0, 60)])
def test_short_requests(m, H, G, D, bands):  # noqa: F811
    both(m, problem([1, 2, 3, 4, 8, 17, 33], [1, 2, 1, 4, 3, 1, 1], H, G, D, 16, seed=bands[0], bands=((120, 127), bands)))


@pytest.mark.parametrize("D", [64, 128])
def test_runs_cut_between_warps_and_ctas(m, D):  # noqa: F811
    # one request on all warps: its pieces' units differ
    both(m, problem([900], [1], 1, 4, D, 64, seed=D, bands=((120, 127), (30, 250))))


@pytest.mark.parametrize("G,D", [(1, 128), (2, 64)])
def test_prompts(m, G, D):  # noqa: F811
    both(m, problem([60, 40, 50, 90], [60, 40, 50, 33], 40, G, D, 32, seed=G, bands=((120, 127), (0, 250))))
