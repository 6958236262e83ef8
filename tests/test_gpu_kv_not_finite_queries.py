"""Query rows with an infinite or NaN element: NaN where they see a key (no finite softmax exists), zeros where they see
none; the other rows as ever."""

import numpy as np
import pytest
import torch

from tests.test_gpu_kv_attention import both, m, problem  # noqa: F401  (m: the fixture)
from tests.test_gpu_kv_queries import key_codes

pytestmark = pytest.mark.gpu

KINDS = [dict(lens=[100, 37, 0, 3], qlens=[1, 3, 1, 5], H=2, G=4, D=128, page=16),
         dict(lens=[90, 1, 40], qlens=[4, 1, 20], H=1, G=7, D=64, page=32),
         dict(lens=[128, 60, 40, 90], qlens=[50, 60, 44, 40], H=40, G=1, D=64, page=64)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("code", [0, 3, 11, None])  # of all keys: zero, positive, negative, any
@pytest.mark.parametrize("scale", [0.2, -0.2, 0.0])
def test_rows_that_are_not_finite(m, kind, value, code, scale):  # noqa: F811
    p = problem(**kind, seed=2)
    rows = np.random.default_rng(1).random(tuple(p["q"].shape[:2])) < 0.3
    q = p["q"].float()
    q[torch.from_numpy(rows)] *= 3e4  # finite elements beyond f16 beside it
    q[..., 37][torch.from_numpy(rows)] = value
    p["q"] = q.to(torch.bfloat16)
    if code is not None:
        key_codes(p, 37, code)
    with np.errstate(invalid="ignore"):
        both(m, p, scale=scale)
