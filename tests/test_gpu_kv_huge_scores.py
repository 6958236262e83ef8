"""Scores up to near the largest float32: a row is the mean of the values of its best keys, its lse their score.

Queries with one element 2^a, keys that differ in that element's code and scale only: every score is exact in float32, best
keys tie exactly, all others weigh nothing (scores differ by 2^15 and more).  Bounds: the result's bf16 rounding and a
weight's, as in test_gpu_kv_attention.py; the lse's factor scale log2 e and back, four roundings of 2^-24 of it.
"""

import numpy as np
import pytest
import torch

from oracle import kv_cache as ref
from tests.test_gpu_kv_attention import m, problem, run  # noqa: F401  (m: the fixture)
from tests.test_gpu_kv_queries import key_codes

pytestmark = pytest.mark.gpu

STREAMED = [dict(lens=[100, 37, 1, 3000], qlens=[1, 3, 1, 1], H=2, G=4, D=128, page=16),
            dict(lens=[90, 500], qlens=[2, 2], H=1, G=16, D=64, page=32)]
PROMPTS = [dict(lens=[300, 128, 520, 90], qlens=[60, 128, 70, 50], H=40, G=1, D=D, page=64) for D in (64, 128)]


def one_element(kind, a, low, high, seed):
    """Keys with codes in element 5 only, scale bytes low .. high."""
    p = problem(**kind, seed=seed, bands=((low, high), (120, 127)))
    p["q"][:] = 0
    p["q"][..., 5] = torch.from_numpy(2.0 ** a * np.random.default_rng(seed).choice([-1, 1], p["q"].shape[:2]))
    codes = p["data"][..., ref.k_at(np.arange(16), 2, p["D"])].copy()
    for j in range(p["D"] // 2):
        p["data"][..., ref.k_at(np.arange(16), j, p["D"])] = 0
    codes = np.where(codes >> 4 & 7, codes, codes | 0x10) & 0xF0  # (no zeros: scores differ)
    p["data"][..., ref.k_at(np.arange(16), 2, p["D"])] = codes
    return p


def compare(p, out, lse, scale):
    kv = [0, p["H"] - 1]
    hq = [h * p["G"] + i for h in kv for i in range(p["G"])]
    want, wl, spread, _ = ref.attention(p["q"].float().numpy()[:, hq], p["data"][:, kv], p["table"], p["lens"], p["start"],
                                        scale)
    got, gl = out.double().cpu().numpy()[:, hq], lse.double().cpu().numpy()[:, hq]
    assert np.isfinite(want).all() and np.abs(wl).max() < 3e38
    bad = ~(np.abs(got - want) <= (2.0 ** -9 + 2.0 ** -13) * (np.abs(want) + spread))
    assert not bad.any(), (bad.mean(), got[bad][:4], want[bad][:4])
    off = ~(np.abs(gl - wl) <= 2.0 ** -22 * np.abs(wl))
    assert not off.any(), (off.mean(), gl[off][:4], wl[off][:4])


@pytest.mark.parametrize("kind", STREAMED + PROMPTS)
@pytest.mark.parametrize("a", [20, 24, 27, 31, 40, 70, 105])
@pytest.mark.parametrize("scale", [1.0, -0.25])
def test_large_queries(m, kind, a, scale):  # noqa: F811
    p = one_element(kind, a, 125, 129, a)
    out, lse = run(m, p, scale)
    compare(p, out, lse, scale)


@pytest.mark.parametrize("kind", STREAMED + PROMPTS[:1])
@pytest.mark.parametrize("a,low,high,scale", [(0, 200, 210, 1.0), (-10, 240, 247, 1.0), (2, 245, 248, 0.5), (-20, 250, 254, -1.0),
                                              (100, 180, 190, 2.0 ** -60)])
def test_large_keys(m, kind, a, low, high, scale):  # noqa: F811
    p = one_element(kind, a, low, high, high)
    out, lse = run(m, p, scale)
    compare(p, out, lse, scale)


@pytest.mark.parametrize("kind", STREAMED + PROMPTS[:1])
@pytest.mark.parametrize("byte", [190, 215, 252])
def test_a_huge_key_after_usual_ones(m, kind, byte):  # noqa: F811
    """One key in the middle of each request is huge: rows of one sign end up on it, the others lose it."""
    p = one_element(kind, 0, 120, 124, byte)
    D, page = p["D"], p["page"]
    for r, n in enumerate(p["lens"]):
        j = n // 2
        p["data"][p["table"][r, j // page], :, j % page // 16, 16 * D + j % 16 * (D // 32)] = byte
    out, lse = run(m, p, 1.0)
    kv = [0, p["H"] - 1]
    hq = [h * p["G"] + i for h in kv for i in range(p["G"])]
    want, wl, spread, _ = ref.attention(p["q"].float().numpy()[:, hq], p["data"][:, kv], p["table"], p["lens"], p["start"], 1.0)
    got, gl = out.double().cpu().numpy()[:, hq], lse.double().cpu().numpy()[:, hq]
    assert (np.abs(wl) > 1e15).any() and (np.abs(wl) < 100).any()
    # usual scores are at most 6 / 8: their products' roundings stay below 2^-20
    light = 2.0 ** -34 * 6 * 1024 if p["H"] == 40 else 0
    bad = ~(np.abs(got - want) <= (2.0 ** -9 + 2.0 ** -13) * (np.abs(want) + spread) + light)
    assert not bad.any(), (bad.mean(), got[bad][:4], want[bad][:4])
    off = ~(np.abs(gl - wl) <= 2.0 ** -20 * (1 + np.abs(wl)))
    assert not off.any(), (off.mean(), gl[off][:4], wl[off][:4])


@pytest.mark.parametrize("kind", STREAMED + PROMPTS)
def test_keys_of_zero_under_the_largest_factor(m, kind):  # noqa: F811
    p = one_element(kind, 126, 120, 127, 5)
    key_codes(p, 5, 0)
    out, lse = run(m, p, 2.0 ** 100)
    compare_zero(p, out, lse)


def compare_zero(p, out, lse):
    """All scores 0: the plain mean of the visible values."""
    q = torch.zeros_like(p["q"])
    want, wl, spread, _ = ref.attention(q.float().numpy()[:, :1], p["data"][:, :1], p["table"], p["lens"], p["start"], 1.0)
    got, gl = out.double().cpu().numpy()[:, :1], lse.double().cpu().numpy()[:, :1]
    assert (np.abs(got - want) <= (2.0 ** -9 + 2.0 ** -13) * (np.abs(want) + spread) + (2.0 ** -34 * 6 * 1024 if p["H"] == 40 else 0)).all()
    assert (np.abs(gl - wl) <= 2.0 ** -20 * (1 + np.abs(wl))).all()
