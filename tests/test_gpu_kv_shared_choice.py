"""Which kernels a call behind a shared prefix takes, asked of the library, and on the tensor cores what the tests of small
batches show on the streaming kernel only: rows of queries that are not finite, beside others and in empty places."""

import ctypes

import numpy as np
import pytest
import torch

from tests import test_gpu_kv_shared as shared
from tests.test_gpu_kv_shared import m  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def slices(m, p):  # noqa: F811
    """Slices that the prefix is cut into on the tensor cores, 0: streamed."""
    n = m._native
    c = n.KvCacheStruct(None, p["pages"], p["page"], p["H"], p["D"])
    N, Hq, D = p["q"].shape
    a = n.KvAttnStruct(len(p["lens"]), N, Hq, p["table"].shape[1], int(np.diff(p["start"]).max()), 1, 0, Hq * D, 1.0)
    return n.load().kv_mxfp4_attention_shared_slices(ctypes.byref(c), ctypes.byref(a), len(p["shared"]))


def long_table(p, tokens=131072):
    """The choice goes by the room of the table, of which a prefix may use little."""
    p["shared"] = np.concatenate([p["shared"], np.full(tokens // p["page"] - len(p["shared"]), -1, np.int32)])
    return p


def test_the_choice(m):  # noqa: F811
    few = shared.problem(300, [5] * 3, [1] * 3, 2, 4, 128, 16)
    assert slices(m, few) == 0
    assert slices(m, shared.problem(16, [5] * 60, [1] * 60, 4, 7, 64, 16)) == 0  # next to no prefix
    many = long_table(shared.problem(300, [5] * 60, [1] * 60, 4, 7, 64, 16))
    assert 1 <= slices(m, many) <= 31
    few["shared"] = np.zeros(0, np.int32)
    assert slices(m, few) == -2
    lib = m._native.load()
    assert lib.kv_mxfp4_attention_shared_slices(None, None, 1) == -1


@pytest.mark.parametrize("kind", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("P", [100, 1500])
@pytest.mark.parametrize("G,D", [(8, 64), (7, 128)])
def test_not_finite_queries(m, kind, P, G, D):  # noqa: F811
    lens = [10, -1, 0] * 14
    p = long_table(shared.problem(P, lens, [1] * 42, 2, G, D, 32, seed=2))
    assert slices(m, p) >= 1
    q = p["q"].clone()
    want = shared.run(m, p)
    shared.check(p, *want)
    for tok, head in ((3, 3), (4, 0), (5, 2 * G - 1)):  # own keys and the prefix; an empty place; the prefix alone
        p["q"][tok, head, 7] = kind
    out, lse = shared.run(m, p)
    assert (out[4] == 0).all() and torch.isneginf(lse[4]).all()
    for tok, head in ((3, 3), (5, 2 * G - 1)):
        assert torch.isnan(out[tok, head]).all() and torch.isnan(lse[tok, head])
        # beside them, as by the oracle: their own rows as they were
        out[tok, head], lse[tok, head] = want[0][tok, head], want[1][tok, head]
    p["q"] = q
    shared.check(p, out, lse)


@pytest.mark.parametrize("P", [100, 1500])
def test_nothing_but_rows_that_are_not_finite(m, P):  # noqa: F811
    p = long_table(shared.problem(P, [10] * 40, [1] * 40, 2, 8, 64, 32, seed=3))
    p["q"][:] = float("nan")
    out, lse = shared.run(m, p)
    assert torch.isnan(out).all() and torch.isnan(lse).all()
