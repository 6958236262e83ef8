"""The parts of a row behind a shared prefix are joined without leaving float32: values near the largest, whose sums over one
part just fit the unit that its keys are counted for, times the number of parts."""

import numpy as np
import pytest
import torch

from oracle import kv_cache as cache
from tests import test_gpu_kv_shared as shared
from tests.test_gpu_kv_shared import m  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
def test_mean_of_one_huge_value(m, D):  # noqa: F811
    """Every value is 1.5 2^127, so every result is.  The scales send the slices to the streaming kernel; the first 16 of every
    128 keys weigh 2^-7.89 of the others (less than would move a row's reference), so weights reach 2^7.89."""
    R, G, P, page = 600, 8, 31 * 128, 128
    p = shared.problem(P, [1] * R, [1] * R, 1, G, D, page, seed=D, extra=0)
    t, byte = np.arange(16), np.arange(D // 2)
    p["data"][..., cache.k_at(t[:, None], byte, D)] = 0
    p["data"][..., cache.k_at(t, 2, D)] = 0x20  # element 5: 1
    p["data"][:, :, 0, :][..., cache.k_at(t, 2, D)] = 0
    p["data"][..., cache.v_at(t[:, None], byte, D)] = 0x77
    p["data"][..., 16 * D:16 * D + D // 2] = 127
    p["data"][..., 16 * D + D // 2:] = 252
    p["q"].zero_()
    p["q"][:, :, 5] = 5.46875
    p["shared"] = np.concatenate([p["shared"], np.zeros(131072 // page - len(p["shared"]), np.int32)])
    out, lse = shared.run(m, p, scale=1.0)
    want = 1.5 * 2.0 ** 127
    assert torch.isfinite(lse).all()
    # weights have 16 bits, the sums of 4000 keys 2^-24 each: within one step of bf16
    assert ((out.double() - want).abs() <= 2.0 ** -8 * want).all(), out.double().unique()[:8]
