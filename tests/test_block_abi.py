"""The attention block's C ABI: every declared symbol is exported by both
libraries, and bad arguments and outputs that share memory with another argument
are refused on the host before any CUDA call."""

import ctypes
import os
import re

import pytest
import torch

from tests.conftest import ROOT

NULL, DIMS, ALIGN, WORKSPACE, OVERLAP = -1, -2, -3, -5, -8


@pytest.fixture(scope="module")
def native():
    from mxfp4_weight_only_gb300 import _native, build

    build.build()
    return _native


def test_declared_symbols_are_exported(native):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "block_mxfp4.h")).read(), flags=re.S)
    names = set(re.findall(r"\b((?:kv|linear)_\w+)\s*\(", text))
    assert {"linear_a16w4_mxfp4", "kv_mxfp4_append_rope"} <= names
    for lib in (native.load(checked=False), native.load(checked=True)):
        for n in names:
            assert n in native.SIGNATURES and hasattr(lib, n), n


# ------------------------------------------------------------------ linear: T = 7, K = 64, N = 48

LINEAR = dict(T=7, K=64, N=48, act=0, out_is_f32=0, x_stride=64, res_stride=48, out_stride=48)
SIZES = dict(x=2 * 7 * 64, w=48 * 32, ws=48 * 2, bias=96, res=2 * 7 * 48, out=2 * 7 * 48, work=256)


def linear(native, at=None, size=256, **kw):
    p = {k: (i + 1) << 20 for i, k in enumerate(SIZES)}
    p.update(at or {})
    d = native.LinearStruct(**{**LINEAR, **kw})
    return native.load().linear_a16w4_mxfp4(ctypes.byref(d), *(p[k] for k in SIZES), size, None)


def test_linear_refusals(native):
    for kw in (dict(T=-1), dict(T=(1 << 24) + 1), dict(K=0), dict(K=48), dict(K=65568, x_stride=65568), dict(N=0), dict(N=(1 << 20) + 1),
               dict(act=-1), dict(act=4), dict(act=3, N=47), dict(out_is_f32=2), dict(x_stride=56), dict(x_stride=68),
               dict(res_stride=47), dict(out_stride=47), dict(T=1 << 24, N=1 << 13, res_stride=1 << 13, out_stride=1 << 13),
               dict(out_stride=(1 << 38) + 1), dict(x_stride=(1 << 38) + 8)):
        assert linear(native, **kw) == DIMS, kw
        d = native.LinearStruct(**{**LINEAR, **kw})
        assert native.load().linear_mxfp4_workspace_bytes(ctypes.byref(d)) == 0
    for k in ("x", "w", "ws", "out", "work"):
        assert linear(native, {k: None}) == NULL, k
    for k, off in (("x", 8), ("w", 8), ("bias", 1), ("res", 1), ("out", 1), ("work", 128)):
        assert linear(native, {k: (1 << 24) + off}) == ALIGN, k
    assert linear(native, {"out": (1 << 24) + 2}, out_is_f32=1) == ALIGN
    assert linear(native, size=255) == WORKSPACE
    assert linear(native, {k: None for k in SIZES}, T=0) == 0
    assert native.load().linear_a16w4_mxfp4(None, *[None] * 7, 0, None) == NULL
    assert native.load().linear_mxfp4_read_status(None, ctypes.byref(ctypes.c_uint32()), None) == NULL


@pytest.mark.parametrize("out", ["out", "work"])
@pytest.mark.parametrize("other", list(SIZES))
def test_linear_overlap(native, out, other):
    if out == other:
        return
    at = {k: (i + 1) << 20 for i, k in enumerate(SIZES)}
    for p in (at[other], at[other] + (SIZES[other] - 1) // 256 * 256):
        if out == "out" and other == "res" and p == at[other]:
            continue  # the residual itself, below
        assert linear(native, {out: p}) == OVERLAP


def test_linear_residual_in_place(native):
    at = {"res": 1 << 24, "out": 1 << 24}
    assert linear(native, at, out_is_f32=1) == OVERLAP
    assert linear(native, at, out_stride=56) == OVERLAP
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only where nothing can be launched")
    assert linear(native, at) == -6


# ------------------------------------------------------------------ rotation and write

ROPE = dict(N=7, Hq=4, x_is_f32=0, rotary_dim=32, interleaved=0, max_positions=9, position_offset=0, q_stride=512, k_stride=512,
            v_stride=512)
ROPE_SIZES = dict(q=2 * (6 * 512 + 256), k=2 * (6 * 512 + 128), v=2 * (6 * 512 + 128), pos=28, slots=28, cs=4 * 9 * 32, q_out=2 * 7 * 256)
CACHE = 3 * 2 * 17 * 64


def rope(native, at=None, cache=None, data=64 << 20, **kw):
    p = {k: (i + 1) << 20 for i, k in enumerate(ROPE_SIZES)}
    p.update(at or {})
    c = native.KvCacheStruct(data, *(cache or (3, 16, 2, 64)))
    r = native.KvRopeStruct(**{**ROPE, **kw})
    return native.load().kv_mxfp4_append_rope(ctypes.byref(c), ctypes.byref(r), *(p[k] for k in ROPE_SIZES), None)


def test_rope_refusals(native):
    for kw in (dict(N=-1), dict(N=(1 << 24) + 1), dict(Hq=-1), dict(Hq=16385, q_stride=16385 * 64), dict(x_is_f32=2), dict(rotary_dim=0),
               dict(rotary_dim=24), dict(rotary_dim=80), dict(interleaved=2), dict(max_positions=0), dict(position_offset=-1),
               dict(q_stride=248), dict(k_stride=120), dict(v_stride=516), dict(x_is_f32=1, k_stride=514), dict(cache=(3, 20, 2, 64))):
        assert rope(native, **kw) == DIMS, kw
    for k in ROPE_SIZES:
        assert rope(native, {k: None}) == NULL, k
    for k, off in (("q", 8), ("k", 8), ("v", 8), ("pos", 2), ("slots", 2), ("cs", 8), ("q_out", 8)):
        assert rope(native, {k: (32 << 20) + off}) == ALIGN, k
    assert rope(native, data=None) == NULL and rope(native, data=(64 << 20) + 8) == ALIGN
    assert rope(native, {k: None for k in ROPE_SIZES}, N=0) == 0
    lib, r = native.load(), native.KvRopeStruct(**ROPE)
    assert lib.kv_mxfp4_append_rope(None, ctypes.byref(r), *[None] * 8) == NULL


@pytest.mark.parametrize("other", ["q", "k", "v", "pos", "slots", "cs", "data"])
def test_rope_overlap(native, other):
    at = {k: (i + 1) << 20 for i, k in enumerate(ROPE_SIZES)}
    if other == "data":
        for p in (64 << 20, (64 << 20) + CACHE - 16, (64 << 20) - ROPE_SIZES["q_out"] + 16):
            assert rope(native, {"q_out": p}) == OVERLAP
        return
    last = at[other] + (ROPE_SIZES[other] - 1) // 16 * 16
    for p in (at[other], last):
        assert rope(native, {"q_out": p}) == OVERLAP
        assert rope(native, data=p) == OVERLAP


# ------------------------------------------------------------------ shared prefix

SHARED_NAMES = ("q", "shared", "len", "table", "lens", "start", "out", "lse", "ws")


def shared(native, at=None, cache=(8, 16, 2, 64), data=64 << 20, size=None, blocks=3, **kw):
    a = native.KvAttnStruct(**{**dict(R=2, N=4, Hq=8, max_blocks=5, max_q_len=2, causal=1, window=0, q_stride=512, scale=0.1), **kw})
    c = native.KvCacheStruct(data, *cache)
    p = {k: (i + 1) << 20 for i, k in enumerate(SHARED_NAMES)}
    p.update(at or {})
    if size is None:
        size = 1 << 40
    return native.load().kv_mxfp4_attention_shared(ctypes.byref(c), ctypes.byref(a), blocks, *(p[k] for k in SHARED_NAMES), size, None)


def shared_workspace(native, blocks=3, **kw):
    a = native.KvAttnStruct(**{**dict(R=2, N=4, Hq=8, max_blocks=5, max_q_len=2, causal=1, window=0, q_stride=512, scale=0.1), **kw})
    c = native.KvCacheStruct(None, 8, 16, 2, 64)
    return native.load().kv_mxfp4_attention_shared_workspace_bytes(ctypes.byref(c), ctypes.byref(a), blocks)


def test_shared_refusals(native):
    for kw in (dict(R=-1), dict(N=-1), dict(Hq=7), dict(max_blocks=0), dict(max_q_len=-1), dict(causal=2), dict(window=4), dict(blocks=0),
               dict(blocks=1 << 27), dict(q_stride=504), dict(scale=float("inf"))):
        assert shared(native, **kw) == DIMS, kw
        assert shared_workspace(native, **kw) == 0, kw
    assert shared(native, cache=(8, 20, 2, 64)) == DIMS
    for k in SHARED_NAMES:
        if k != "lse":
            assert shared(native, {k: None}) == NULL, k
    for k, off in (("q", 8), ("shared", 2), ("len", 2), ("table", 2), ("lens", 2), ("start", 2), ("out", 8), ("lse", 2), ("ws", 128)):
        assert shared(native, {k: (32 << 20) + off}) == ALIGN, k
    need = shared_workspace(native)
    assert need > 0 and shared(native, size=need - 1) == WORKSPACE
    for kw in (dict(R=0), dict(N=0), dict(max_q_len=0)):
        assert shared(native, {k: None for k in SHARED_NAMES}, **kw) == 0


def test_shared_overlap(native):
    size = dict(q=2 * 4 * 512, shared=12, len=4, table=40, lens=8, start=12, data=8 * 2 * 17 * 64, out=2 * 4 * 512, lse=4 * 32,
                ws=shared_workspace(native))
    at = {k: (i + 1) << 24 for i, k in enumerate(size)}
    for out in ("out", "lse", "ws"):
        for other in size:
            if out == other:
                continue
            for p in (at[other], at[other] + (size[other] - 1) // 256 * 256):
                x = {**at, out: p}
                data = x.pop("data")
                assert shared(native, x, data=data, size=size["ws"]) == OVERLAP, (out, other)


def test_shared_workspace_grows_with_rows_and_slices(native):
    few, many = shared_workspace(native, N=2), shared_workspace(native, N=64, R=64)
    assert many - few >= (64 - 2) * 8 * 64 * 4 * 2
    assert shared_workspace(native, N=64, R=64, blocks=4000) > many
