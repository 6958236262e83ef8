"""Queries whose elements are of very unlike size, against keys that make the small ones count.

The kernels hold a row's queries as f16 times a power of two and look after rows where that loses bits that could move a
score by more than 2^-16 (units of log2): the bounds of test_gpu_kv_attention.py with 2^-16 ln 2 < 2^-16 more in each score,
    |out - ref| <= ... + 2 * 2^-16 spread,   |lse - ref| <= ... + 2^-16.
"""

import numpy as np
import pytest
import torch

from oracle import kv_cache as ref
from tests.test_gpu_kv_attention import m, problem, run  # noqa: F401  (m: the fixture)

pytestmark = pytest.mark.gpu

STREAMED = [dict(lens=[100, 37, 1, 300], qlens=[1, 3, 1, 2], H=2, G=G, D=D, page=16) for G, D in ((4, 128), (7, 64), (16, 128))]
# rows above 32 with a request and head for every SM: the tensor-core kernel, up to 256 keys and more
PROMPTS = [dict(lens=[300, 128, 520, 90], qlens=[60, 128, 70, 50], H=40, G=1, D=D, page=64) for D in (64, 128)]
KINDS = STREAMED + PROMPTS


def compare(p, out, lse, scale):
    kv = [0, p["H"] - 1]
    hq = [h * p["G"] + i for h in kv for i in range(p["G"])]
    want, wl, spread, size = ref.attention(p["q"].float().numpy()[:, hq], p["data"][:, kv], p["table"], p["lens"], p["start"],
                                           scale)
    got, gl = out.double().cpu().numpy()[:, hq], lse.double().cpu().numpy()[:, hq]
    D = p["D"]
    err = D * 2.0 ** -24 * size + 2.0 ** -16
    # (prompts that see more than 256 keys: half of f16's step in units of 2^-9 of the values' sum)
    light = 2.0 ** -34 * 6 * 1024 if p["H"] == 40 else 0
    bound = (2.0 ** -9 + 2.0 ** -13) * np.abs(want) + (2.0 ** -9 + 2.0 ** -13 + 2 * err[..., None]) * spread + light
    assert np.isfinite(want).all()
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (bad.mean(), got[bad][:4], want[bad][:4], bound[bad][:4])
    off = ~(np.abs(gl - wl) <= err + 2.0 ** -20 * (1 + np.abs(wl)))
    assert not off.any(), (off.mean(), gl[off][:4], wl[off][:4])


def key_codes(p, element, code):
    """Every key's code of one element."""
    D = p["D"]
    for t in range(16):
        at = ref.k_at(t, element // 2, D)
        old = p["data"][..., at]
        p["data"][..., at] = old & 0xF0 | code if element % 2 == 0 else old & 0x0F | code << 4


def key_scales(p, block, low, high, seed=0):
    D = p["D"]
    NB = D // 32
    at = 16 * D + block + NB * np.arange(16)
    p["data"][..., at] = np.random.default_rng(seed).integers(low, high + 1, p["data"][..., at].shape)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("power", [18, 22, 24, 31, 40, 90])
def test_one_large_element_under_keys_without_it(m, kind, power):  # noqa: F811
    # the element's own code is zero in every key; the rest of its block is not
    p = problem(**kind, seed=power)
    p["q"][:, :, 5] = 2.0 ** power
    key_codes(p, 5, 0)
    out, lse = run(m, p, 0.3)
    compare(p, out, lse, 0.3)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("power", [20, 26, 35, 60])
def test_blocks_of_unlike_size_against_opposite_keys(m, kind, power):  # noqa: F811
    p = problem(**kind, seed=power)
    p["q"][:, :, :32] *= 2.0 ** power
    key_scales(p, 0, 124 - power, 126 - power)
    out, lse = run(m, p, 0.3)
    compare(p, out, lse, 0.3)


@pytest.mark.parametrize("kind", KINDS)
def test_a_few_rows_of_many(m, kind):  # noqa: F811
    # large elements in some rows and heads only, keys without them in some tokens only
    p = problem(**kind, seed=3)
    g = np.random.default_rng(4)
    N, Hq, D = p["q"].shape
    some = torch.from_numpy(g.random((N, Hq)) < 0.1)
    p["q"][..., D - 1] = torch.where(some, torch.tensor(2.0 ** 23), p["q"][..., D - 1].float()).to(torch.bfloat16)
    key_codes(p, D - 1, 8)  # -0
    out, lse = run(m, p, 0.3)
    compare(p, out, lse, 0.3)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("qexp,kexp,scale", [(-100, 98, 1.0), (100, -110, 2.0), (-120, 60, 2.0 ** 60), (60, 0, -2.0 ** -62),
                                             (-126, 120, 3.0), (0, 127, 2.0 ** -126)])
def test_whole_rows_of_any_size(m, kind, qexp, kexp, scale):  # noqa: F811
    p = problem(**kind, seed=8, bands=((127 + kexp - 1, 127 + kexp - 1), (120, 127)))
    p["q"] = (p["q"].double() * 2.0 ** qexp).to(torch.bfloat16)
    out, lse = run(m, p, scale)
    compare(p, out, lse, scale)


@pytest.mark.parametrize("kind", KINDS)
def test_zero_scale_and_zero_rows(m, kind):  # noqa: F811
    p = problem(**kind, seed=9)
    out, lse = run(m, p, 0.0)
    compare(p, out, lse, 0.0)
    p["q"][::2] = 0
    out, lse = run(m, p, -0.3)
    compare(p, out, lse, -0.3)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("large,small,keys,scale", [(120, -128, 250, 0.5), (110, -40, 163, 0.5), (60, -126, 252, 2.0)])
def test_elements_that_vanish_beside_the_largest(m, kind, large, small, keys, scale):  # noqa: F811
    # more than 2^149 below it: nothing is left of them in float32 after the row's power of two either
    p = problem(**kind, seed=11, bands=((keys, keys), (120, 127)))
    p["q"] = (p["q"].double() * 2.0 ** small).to(torch.bfloat16)
    p["q"][:, :, 5] = 2.0 ** large
    key_codes(p, 5, 0)
    out, lse = run(m, p, scale)
    compare(p, out, lse, scale)
