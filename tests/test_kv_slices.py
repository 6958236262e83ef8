"""How the keys of a long request are cut (functions of csrc/kv_internal.h, compiled for the host), up to the longest that a call
takes.  Slices of a shared prefix cover its keys once, in order, each but the first beginning at a multiple of 128; the
tensor-core kernel's tiles are those that hold a key, and whole where every key of them is seen."""

import ctypes
import os
import subprocess

import pytest

from mxfp4_weight_only_gb300 import build
from tests.conftest import ROOT

SOURCE = """#include "kv_internal.h"
extern "C" void slice(int P, int splits, int i, int* base, int* n) {
  const moe::KvSlice s = moe::kv_slice(P, splits, i);
  *base = s.base;
  *n = s.n;
}
extern "C" int tiles(int lo, int hi) { return moe::kv_tiles(lo, hi); }
extern "C" int whole(int lo, int hi, int j0) { return moe::kv_whole_tile(lo, hi, j0); }
extern "C" int max_splits() { return moe::kMaxSplits; }
extern "C" int slice_keys() { return moe::kSliceKeys; }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("slices")
    (d / "slices.cu").write_text(SOURCE)
    r = subprocess.run([build.nvcc()] + build.FLAGS + ["-I" + os.path.join(ROOT, "mxfp4_weight_only_gb300", "csrc"), "-shared",
                                                       "-o", str(d / "slices.so"), str(d / "slices.cu")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return ctypes.CDLL(str(d / "slices.so"))


LONG = [2 ** 31 - 1 - k for k in range(131)] + [2 ** 31 - 1 - 128 * k for k in range(2, 66)] + [2 ** 30, 2 ** 30 + 1]
SHORT = list(range(300)) + [128 * 31 + k for k in (-1, 0, 1)] + [4000, 100003, 10 ** 6]


@pytest.mark.parametrize("lengths", [SHORT, LONG])
def test_slices_cover_the_prefix(lib, lengths):
    base, n = ctypes.c_int(), ctypes.c_int()
    unit = lib.slice_keys()
    for P in lengths:
        for splits in range(1, lib.max_splits() + 1):
            at, first = 0, None
            for i in range(splits):
                lib.slice(P, splits, i, ctypes.byref(base), ctypes.byref(n))
                assert base.value == at and n.value >= 0, (P, splits, i, base.value, n.value)
                first = n.value if first is None else first
                # all alike but the last that has any
                assert n.value == first or at + n.value == P
                assert n.value == 0 or at % unit == 0
                at += n.value
            assert at == P, (P, splits, at)


def test_tiles_of_keys(lib):
    edges = [0, 1, 127, 128, 129, 255, 256, 1000, 2 ** 30] + [2 ** 31 - 1 - k for k in (0, 1, 15, 16, 17, 126, 127, 128, 255, 256, 300)]
    for lo in edges:
        for hi in edges:
            want = (hi - 1) // 128 - lo // 128 + 1 if hi > lo else 0
            assert lib.tiles(lo, hi) == want, (lo, hi)
            for j0 in {lo // 128 * 128, hi // 128 * 128, max(hi - 1, 0) // 128 * 128}:
                assert bool(lib.whole(lo, hi, j0)) == (lo <= j0 and j0 + 128 <= hi), (lo, hi, j0)
