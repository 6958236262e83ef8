"""Page tables at counts near 2^31 (18 GB of device memory): the token index steps past the largest int, a request's length
would, and finished requests claim more pages than an int counts."""

import numpy as np
import pytest
import torch

from oracle import kv_cache as ref
from tests.test_gpu_kv_attention import i32, m  # noqa: F401  (m: the fixture)

pytestmark = pytest.mark.gpu


def test_the_most_tokens(m):  # noqa: F811
    M = 2 ** 31 - 1
    table, ring = np.array([[7, -1, -1], [3, 4, -1]], np.int32), np.arange(20, dtype=np.int32)
    bt, rg = i32(table), i32(ring)
    got = m.kv_page_tables(i32([5, 30]), i32([20, 3]), bt, rg, i32([18, 9]), 16, M)
    seq, start, slots, pos, state = ref.page_tables([5, 30], [20, 3], table, ring, [18, 9], 16, 40)
    assert got.seq_lens.tolist() == seq.tolist() and got.query_start.tolist() == start.tolist()
    assert got.ring_state.tolist() == state.tolist() and np.array_equal(bt.cpu().numpy(), table)
    assert got.slots[:40].tolist() == slots.tolist() and got.positions[:40].tolist() == pos.tolist()
    for x in (got.slots, got.positions):
        for i in range(40, M, 2 ** 28):
            assert (x[i: i + 2 ** 28] == -1).all(), i


def test_a_request_past_the_longest_is_refused(m):  # noqa: F811
    page, mb = 256, 2 ** 23 + 1
    cached, new = [2 ** 31 - 10, 2 ** 31 - 10, 5], [20, 9, 3]
    table = np.zeros((3, mb), np.int32)
    table[1, -2], table[2, 0] = 3, 1
    ring = np.array([5, 6], np.int32)
    bt, rg = i32(table), i32(ring)
    got = m.kv_page_tables(i32(cached), i32(new), bt, rg, i32([0, 2]), page, 40)
    want = ref.page_tables(cached, new, table, ring, [0, 2], page, 40)
    assert want[0].tolist() == [-1, 2 ** 31 - 1, 8]
    for name, a, b in zip(got._fields, got, want):
        assert np.array_equal(a.cpu().numpy(), b), name
    assert np.array_equal(bt.cpu().numpy(), table)


def test_more_pages_given_back_than_the_ring_holds_stay_inside_it(m):  # noqa: F811
    R, mb, C = 17, 2 ** 27, 1000
    around = torch.full((3 * C,), 77, dtype=torch.int32, device="cuda")
    table = torch.full((R, mb), 5, dtype=torch.int32, device="cuda")
    got = m.kv_page_tables(i32([2 ** 31 - 1] * R), i32([-1] * R), table, around[C: 2 * C], i32([3, 4]), 16, 100000)
    assert got.seq_lens.tolist() == [0] * R and (got.slots == -1).all()
    assert (around[:C] == 77).all() and (around[2 * C:] == 77).all() and (around[C: 2 * C] == 5).all()
