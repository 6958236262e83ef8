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
