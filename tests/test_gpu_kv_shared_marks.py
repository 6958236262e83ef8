"""Rows whose results a call behind a shared prefix throws away (empty places of the batch, rows before the first request, past
the last or past max_q_len) cost nothing: where they hold what the tensor cores cannot, the other rows' results are bit for bit
those beside rows of zeros.

On the tensor cores a slice with rows that f16 cannot hold (not finite, elements of very unlike size, of a size that its factor
leaves the range) is done over by the streaming kernel, which takes three times as long and rounds otherwise: the bits show that
it was not."""

import numpy as np
import pytest
import torch

from tests import test_gpu_kv_shared as shared
from tests.test_gpu_kv_shared import m  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

KINDS = ["nan", "inf", "unlike", "huge"]


def spoil(q, rows, kind):
    q = q.clone()
    if kind == "unlike":
        q[rows] = 1.5 * 2.0 ** -20  # 2^-26 in f16 beside 2^20
        q[rows, :, 3] = 2.0 ** 20
    else:
        q[rows] = {"nan": float("nan"), "inf": float("inf"), "huge": 2.0 ** 120}[kind]
    return q


def long_table(p):
    g = np.random.default_rng(1)
    tail = g.integers(-5, p["pages"] + 5, 131072 // p["page"] - len(p["shared"])).astype(np.int32)
    p["shared"] = np.concatenate([p["shared"], tail])
    return p


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G,D", [(8, 64), (7, 128)])
def test_empty_places(m, kind, G, D):  # noqa: F811
    lens = [20, -1] * 30
    p = long_table(shared.problem(1500, lens, [1] * 60, 2, G, D, 64, seed=G))
    shared.both(m, p)
    p["q"][1::2] = 0
    want = shared.run(m, p)
    q = p["q"].clone()
    p["q"] = spoil(q, slice(1, None, 2), kind)
    got = shared.run(m, p)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # (a row that counts does change what is done)
    p["q"] = spoil(q, slice(2, 3), kind)
    got = shared.run(m, p)
    assert not torch.equal(got[0][4:], want[0][4:])


@pytest.mark.parametrize("kind", KINDS)
def test_rows_of_no_request(m, kind):  # noqa: F811
    p = long_table(shared.problem(1500, [9] * 41, [9] * 41, 2, 8, 64, 64, seed=3, gaps=4))
    # the first request's rows belong to none
    p["lens"], p["start"], p["table"] = p["lens"][1:], p["start"][1:], p["table"][1:]
    first = int(p["start"][0])
    used = torch.zeros(p["q"].shape[0], dtype=torch.bool)
    for s in p["start"][:-1]:
        used[s: s + 4] = True
    assert not used[:first].any()
    p["q"][~used] = 0
    want = shared.run(m, p, max_q=4)
    p["q"] = spoil(p["q"], ~used, kind)
    got = shared.run(m, p, max_q=4)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
