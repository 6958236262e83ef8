"""The 4-bit KV cache's C ABI: every declared symbol is exported by both
libraries, and bad arguments are refused on the host before any CUDA call."""

import ctypes
import os
import re

import pytest

from tests.conftest import ROOT


@pytest.fixture(scope="module")
def native():
    from mxfp4_weight_only_gb300 import _native, build

    build.build()
    return _native


def test_declared_symbols_are_exported(native):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "kv_mxfp4.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(kv_mxfp4_\w+)\s*\(", text))
    assert len(names) == 7
    for lib in (native.load(checked=False), native.load(checked=True)):
        for n in names:
            assert n in native.SIGNATURES and hasattr(lib, n), n


def cache(native, data=16, pages=8, page=64, heads=4, D=128):
    return native.KvCacheStruct(data, pages, page, heads, D)


def test_cache_sizes(native):
    lib = native.load()
    size = lambda **kw: lib.kv_mxfp4_cache_bytes(ctypes.byref(cache(native, **kw)))  # noqa: E731
    assert size() == 8 * 4 * 4 * 17 * 128
    assert size(page=16, D=64, heads=1, pages=1) == 17 * 64
    assert size(pages=1 << 20, heads=256) == (1 << 20) * 256 * 4 * 17 * 128  # above 32 bits
    for bad in (dict(page=8), dict(page=48), dict(page=512), dict(pages=0), dict(heads=0), dict(heads=257),
                dict(D=96), dict(D=256), dict(pages=1 << 25)):
        assert size(**bad) == 0, bad


def test_page_table_refusals(native):
    lib, p = native.load(), ctypes.c_void_p(16)

    def call(R=4, page=16, mb=8, mt=64, C=32, ptrs=None, **kw):
        ptrs = [p] * 10 if ptrs is None else ptrs
        return lib.kv_mxfp4_page_tables(R, page, mb, mt, C, *ptrs, None)

    for kw in (dict(R=-1), dict(R=8193), dict(page=24), dict(mb=0), dict(mt=-1), dict(C=0)):
        assert call(**kw) == -2, kw
    for i in range(10):
        assert call(ptrs=[None if k == i else p for k in range(10)]) == -1, i
        assert call(ptrs=[ctypes.c_void_p(18) if k == i else p for k in range(10)]) == -3, i


def test_append_and_gather_refusals(native):
    lib, p = native.load(), ctypes.c_void_p(16)

    def append(c=None, k=p, v=p, f32=0, ks=512, vs=512, N=4, slots=p):
        return lib.kv_mxfp4_append(ctypes.byref(c or cache(native)), k, v, f32, ks, vs, N, slots, None)

    assert lib.kv_mxfp4_append(None, p, p, 0, 512, 512, 4, p, None) == -1
    for kw in (dict(c=cache(native, page=20)), dict(f32=2), dict(N=-1), dict(N=(1 << 24) + 1), dict(ks=504),
               dict(vs=516), dict(f32=1, ks=514)):
        assert append(**kw) == -2, kw
    for kw in (dict(c=cache(native, data=None)), dict(k=None), dict(v=None), dict(slots=None)):
        assert append(**kw) == -1, kw
    for kw in (dict(c=cache(native, data=8)), dict(k=ctypes.c_void_p(24)), dict(slots=ctypes.c_void_p(2))):
        assert append(**kw) == -3, kw
    assert append(N=0, k=None, v=None, slots=None) == 0

    def gather(c=None, slots=p, N=4, k=p, v=p):
        return lib.kv_mxfp4_gather(ctypes.byref(c or cache(native)), slots, N, k, v, None)

    assert lib.kv_mxfp4_gather(None, p, 4, p, p, None) == -1
    assert gather(c=cache(native, heads=300)) == -2 and gather(N=-1) == -2
    assert gather(slots=None) == -1 and gather(k=None) == -1 and gather(v=ctypes.c_void_p(8)) == -3
    assert gather(N=0, slots=None, k=None, v=None) == 0


def test_attention_refusals(native):
    lib, p, w = native.load(), ctypes.c_void_p(16), ctypes.c_void_p(256)

    def call(c=None, q=p, bt=p, sl=p, qs=p, out=p, lse=None, ws=w, size=1 << 40, **kw):
        a = dict(R=2, N=4, Hq=28, max_blocks=4, max_q_len=2, causal=1, window=0, q_stride=28 * 128, scale=0.1)
        a.update(kw)
        return lib.kv_mxfp4_attention(ctypes.byref(c or cache(native)), ctypes.byref(native.KvAttnStruct(**a)), q, bt,
                                      sl, qs, out, lse, ws, size, None)

    for kw in (dict(R=-1), dict(R=65536), dict(N=-1), dict(N=(1 << 24) + 1), dict(Hq=0), dict(Hq=30), dict(Hq=260, q_stride=260 * 128),
               dict(max_blocks=0), dict(max_blocks=1 << 26), dict(max_q_len=-1), dict(causal=2), dict(window=-1),
               dict(window=4, causal=0), dict(q_stride=28 * 128 - 8), dict(q_stride=28 * 128 + 4),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(c=cache(native, D=32))):
        assert call(**kw) == -2, kw
    for kw in (dict(q=None), dict(bt=None), dict(sl=None), dict(qs=None), dict(out=None), dict(ws=None),
               dict(c=cache(native, data=None))):
        assert call(**kw) == -1, kw
    for kw in (dict(q=ctypes.c_void_p(8)), dict(out=ctypes.c_void_p(8)), dict(ws=p), dict(lse=ctypes.c_void_p(2))):
        assert call(**kw) == -3, kw
    assert call(size=16) == -5
    for kw in (dict(R=0), dict(N=0), dict(max_q_len=0)):
        assert call(q=None, out=None, ws=None, **kw) == 0, kw
    a = native.KvAttnStruct(2, 4, 28, 4, 2, 1, 0, 28 * 128, 0.1)
    assert lib.kv_mxfp4_attention_workspace_bytes(ctypes.byref(cache(native)), ctypes.byref(a)) >= 256
    a.Hq = 27
    assert lib.kv_mxfp4_attention_workspace_bytes(ctypes.byref(cache(native)), ctypes.byref(a)) == 0
    assert lib.kv_mxfp4_read_status(None, ctypes.byref(ctypes.c_uint32()), None) == -1
