"""Outputs that share memory with another argument are refused on the host: the kernels' CTAs read their inputs while
others write, in no order."""

import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def native():
    from mxfp4_weight_only_gb300 import _native, build

    build.build()
    return _native


OVERLAP = -8
# kv_mxfp4_page_tables: R = 4, max_blocks = 8, max_tokens = 64, ring of 32
TABLES = dict(cached=16, new=16, table=128, ring=128, state=8, seq=16, start=20, slots=256, positions=256, state_out=8)


@pytest.mark.parametrize("out", ["table", "ring", "seq", "start", "slots", "positions", "state_out"])
@pytest.mark.parametrize("other", list(TABLES))
def test_page_tables(native, out, other):
    if out == other:
        return
    lib = native.load()

    def call(at):
        return lib.kv_mxfp4_page_tables(4, 16, 8, 64, 32, *(ctypes.c_void_p(at[k]) for k in TABLES), None)

    at = {k: 4096 * (i + 1) for i, k in enumerate(TABLES)}
    last = at[other] + TABLES[other] - 4
    for p in (at[other], last, at[other] + 4 - TABLES[out]):  # the same start, the other's last entry, its first
        assert call({**at, out: p}) == OVERLAP
    assert native.ERRORS[OVERLAP] == "MOE_ERR_OVERLAP"
    assert b"shares memory" in lib.moe_error_string(OVERLAP)


@pytest.mark.parametrize("other", list(TABLES))
def test_neighbours_and_shared_inputs_are_taken(native, other):
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only where nothing can be launched")
    lib = native.load()
    at = {k: 4096 * (i + 1) for i, k in enumerate(TABLES)}
    if other != "seq":
        at["seq"] = at[other] + TABLES[other]
    at["new"] = at["cached"]
    assert lib.kv_mxfp4_page_tables(4, 16, 8, 64, 32, *(ctypes.c_void_p(at[k]) for k in TABLES), None) == -6


# 2 requests, 4 rows of 8 heads over 2 kv heads of 64, a cache of 3 pages of 16 tokens
CACHE = 3 * 2 * 17 * 64


def attention_args(native):
    a = native.KvAttnStruct(2, 4, 8, 5, 2, 1, 0, 8 * 64, 0.1)
    ws = native.load().kv_mxfp4_attention_workspace_bytes(
        ctypes.byref(native.KvCacheStruct(None, 3, 16, 2, 64)), ctypes.byref(a))
    return a, dict(q=2 * 4 * 8 * 64, table=4 * 2 * 5, lens=8, start=12, data=CACHE, out=2 * 4 * 8 * 64, lse=4 * 4 * 8, ws=ws)


@pytest.mark.parametrize("out", ["out", "lse", "ws"])
@pytest.mark.parametrize("other", ["q", "table", "lens", "start", "data", "out", "lse", "ws"])
def test_attention(native, out, other):
    if out == other:
        return
    a, size = attention_args(native)

    def call(at):
        c = native.KvCacheStruct(at["data"], 3, 16, 2, 64)
        p = {k: ctypes.c_void_p(v) for k, v in at.items()}
        return native.load().kv_mxfp4_attention(ctypes.byref(c), ctypes.byref(a), p["q"], p["table"], p["lens"],
                                                p["start"], p["out"], p["lse"], p["ws"], size["ws"], None)

    at = {k: (i + 1) << 24 for i, k in enumerate(size)}
    inside = (size[other] - 1) // 256 * 256
    for p in (at[other], at[other] + inside):
        assert call({**at, out: p}) == OVERLAP


@pytest.mark.parametrize("which", ["k", "v", "slots"])
def test_append(native, which):
    at = dict(k=1 << 20, v=2 << 20, slots=3 << 20)
    # rows 512 elements apart: 7 rows of 128 end 3200 elements on
    end = dict(k=2 * (6 * 512 + 128), v=2 * (6 * 512 + 128), slots=28)[which]
    for data in (at[which], at[which] + (end - 1) // 16 * 16, at[which] - CACHE + 16):
        c = native.KvCacheStruct(data, 3, 16, 2, 64)
        assert native.load().kv_mxfp4_append(ctypes.byref(c), at["k"], at["v"], 0, 512, 512, 7, at["slots"], None) == OVERLAP


def test_gather(native):
    c = native.KvCacheStruct(1 << 20, 3, 16, 2, 64)

    def call(slots=2 << 20, k=3 << 20, v=4 << 20):
        return native.load().kv_mxfp4_gather(ctypes.byref(c), slots, 7, k, v, None)

    rows = 2 * 7 * 128
    for kw in (dict(k=1 << 20), dict(v=(1 << 20) + CACHE - 16), dict(k=4 << 20), dict(k=(4 << 20) + rows - 16),
               dict(v=2 << 20), dict(slots=(3 << 20) + rows - 4)):
        assert call(**kw) == OVERLAP


@pytest.mark.gpu
def test_lengths_in_place_are_refused_through_the_binding(native):
    import mxfp4_weight_only_gb300 as m

    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, new, table, ring, state = i32([3, 0]), i32([1, 2]), i32([[0, 1], [2, 3]]), i32([4, 5]), i32([0, 2])
    for kw in (dict(seq_lens=lens), dict(slots=new), dict(positions=ring), dict(query_start=table.view(-1)[:3])):
        with pytest.raises(m.MoeError, match="OVERLAP"):
            m.kv_page_tables(lens, new, table, ring, state, 16, 2, **kw)
    assert m.kv_page_tables(lens, new, table, ring, state, 16, 4).seq_lens.tolist() == [4, 2]
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_results_over_queries_are_refused_through_the_binding(native):
    import mxfp4_weight_only_gb300 as m

    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    c = m.KvCacheMxfp4(3, 16, 2, 64, data=torch.zeros(3, 2, 1, 17 * 64, dtype=torch.uint8, device="cuda"))
    q = torch.randn(4, 8, 64, device="cuda").bfloat16()
    args = (q, c, i32([[0, 1], [2, 0]]), i32([20, 9]), i32([0, 2, 4]), 2)
    with pytest.raises(m.MoeError, match="OVERLAP"):
        m.attention_kv_mxfp4(*args, out=q)
    k, v = torch.empty(2, 3, 2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(m.MoeError, match="OVERLAP"):
        m.kv_gather_mxfp4(c, i32([0, 1, 2]), k_out=k, v_out=k)
    m.attention_kv_mxfp4(*args)
    m.kv_gather_mxfp4(c, i32([0, 1, 2]), k_out=k, v_out=v)
    torch.cuda.synchronize()
