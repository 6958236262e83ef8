"""Attention behind a shared prefix on the tensor cores: the cases of tests/test_gpu_kv_shared.py with 256 rows or more a
kv head (a tail of short requests) and a shared table of 131,072 tokens, most of whose entries, all of them garbage, lie past
the prefix.  The choice between the two kernels goes by the rows and the table, so that short prefixes get here too."""

import numpy as np
import pytest
import torch

from tests import test_gpu_kv_shared as shared
from tests.test_gpu_kv_shared import (  # noqa: F401
    m, test_bad_pages_are_invisible, test_batches, test_decode, test_equal_scores_across_the_parts,
    test_huge_scores, test_long_prefix_is_cut, test_many_requests, test_nan_tokens, test_negative_and_zero_scale,
    test_page_sizes, test_prompts_behind_a_prefix, test_scales_of_any_size, test_several_query_rows)

pytestmark = pytest.mark.gpu

_problem = shared.problem


@pytest.fixture(autouse=True)
def many_rows(monkeypatch):
    """Problems with a long table and, but for tests that count their requests, a tail of requests of two rows."""
    def problem(P, lens, qlens, H, G, D, page, seed=0, **kw):
        if not problem.exact:
            n = -(-256 // (2 * G))
            lens, qlens = list(lens) + [5] * n, list(qlens) + [2] * n
        p = _problem(P, lens, qlens, H, G, D, page, seed=seed, **kw)
        g = np.random.default_rng(seed)
        tail = g.integers(-5, p["pages"] + 5, 131072 // page - len(p["shared"])).astype(np.int32)
        p["shared"] = np.concatenate([p["shared"], tail])
        return p

    problem.exact = False
    monkeypatch.setattr(shared, "problem", problem)
    return problem


@pytest.mark.parametrize("R", [40, 130])
def test_captured(many_rows, m, R):  # noqa: F811
    many_rows.exact = True
    shared.test_captured_and_repeatable(m, R)


def test_the_rows_used_fewer(m):  # noqa: F811
    """A padded batch: the call's N is of 256 rows and more, the requests' of a few."""
    p = shared.problem(700, [40, 3], [1, 1], 4, 7, 64, 32)
    p["lens"], p["start"], p["table"] = p["lens"][:2], p["start"][:3], p["table"][:2]
    shared.both(m, p)


def test_strided_queries(m):  # noqa: F811
    p = shared.problem(400, [24] * 12, [1] * 12, 2, 4, 128, 16, seed=7)
    N = p["q"].shape[0]
    wide = torch.full((N, 14, 128), 1e30, dtype=torch.bfloat16, device="cuda")
    wide[:, :8] = p["q"].cuda()
    shared.both(m, p, q=wide[:, :8], stream=torch.cuda.Stream())


def test_nothing_to_see(many_rows, m):  # noqa: F811
    shared.both(m, shared.problem(0, [0, -1, 3, 0], [2, 1, 1, 20], 2, 4, 64, 16))
    many_rows.exact = True
    out, lse = shared.run(m, shared.problem(100, [-1] * 70, [1] * 70, 2, 4, 64, 16))
    assert (out == 0).all() and torch.isinf(lse).all()
