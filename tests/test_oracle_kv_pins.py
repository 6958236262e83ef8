"""Pins of the 4-bit KV cache oracle: the record layout is a bijection, the
write inverts the read, the quantiser's corner cases, the attention against a
dense torch float64 formulation, the page tables' invariants."""

import numpy as np
import pytest
import torch

from oracle import formats, kv_cache


@pytest.mark.parametrize("D", [64, 128])
def test_record_layout_is_a_bijection(D):
    t, j = np.meshgrid(np.arange(16), np.arange(D // 2), indexing="ij")
    at = np.concatenate([kv_cache.k_at(t, j, D).ravel(), kv_cache.v_at(t, j, D).ravel()])
    assert sorted(at) == list(range(16 * D))
    # spot values of the documented order: K [half][g][t][NB][4], V [hi][g][t][lo][NB][2]
    NB = D // 32
    assert kv_cache.k_at(9, 16 + 7, D) == ((1 * 8 + 1) * 4 + 1) * NB * 4 + 4 + 3
    assert kv_cache.v_at(13, 16 + 5, D) == 8 * D + (((1 * 8 + 2) * 4 + 2) * 2 + 1) * NB * 2 + 2 + 1


def test_write_then_read_round_trips():
    g = np.random.default_rng(0)
    D, H, p = 64, 3, 32
    data = g.integers(0, 256, (4, H, p // 16, 17 * D), dtype=np.uint8)
    x = g.standard_normal((2, 5, H, D))
    slots = np.array([0, 17, 33, 127, 64])
    kc, ks = kv_cache.quantize(x[0])
    vc, vs = kv_cache.quantize(x[1])
    for i, s in enumerate(slots):
        for h in range(H):
            kv_cache.write(data, s, h, kc[i, h], ks[i, h], vc[i, h], vs[i, h])
    for a, b in zip(kv_cache.read(data, slots), (kc, ks, vc, vs)):
        assert np.array_equal(a, b)


def test_quantiser_of_nan_and_infinity():
    x = np.zeros((3, 64))
    x[0, 3] = np.nan
    x[1, 40], x[1, 41], x[1, 42] = np.inf, -np.inf, -(2.0 ** 126)
    x[2, 0] = 1.0
    c, s = kv_cache.quantize(x)
    assert s.tolist() == [[255, 0], [0, 252], [125, 0]]
    u = formats.unpack_nibbles(c)
    assert u[1, 40:43].tolist() == [7, 15, 12] and u[2, 0] == 6  # 1 = 4 * 2^-2


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 5), (False, 0)])
def test_attention_matches_dense_torch(causal, window):
    g = np.random.default_rng(1)
    D, H, Hq, p = 64, 2, 6, 16
    lens, qs = [23, 0, 7, 3], [0, 4, 6, 7, 12]  # the last request has more rows than keys
    table = g.permutation(12).reshape(4, 3).astype(np.int32)
    data = np.zeros((12, H, 1, 17 * D), np.uint8)
    data[..., :16 * D] = g.integers(0, 256, data[..., :16 * D].shape)
    data[..., 16 * D:] = g.integers(120, 128, data[..., 16 * D:].shape)
    q = g.standard_normal((12, Hq, D))
    out, lse, _, _ = kv_cache.attention(q, data, table, np.array(lens), np.array(qs), 0.3, causal, window)
    for r, n in enumerate(lens):
        rows = slice(qs[r], qs[r + 1])
        ql = qs[r + 1] - qs[r]
        j = np.arange(n)
        kc, ks, vc, vs = kv_cache.read(data, table[r, j // p] * p + j % p)
        k = torch.from_numpy(kv_cache.values(kc, ks)).repeat_interleave(Hq // H, 1)
        v = torch.from_numpy(kv_cache.values(vc, vs)).repeat_interleave(Hq // H, 1)
        s = torch.einsum("ihd,jhd->hij", torch.from_numpy(q[rows]), k) * 0.3
        pos = torch.arange(ql)[:, None] + n - ql
        see = torch.ones(ql, n, dtype=torch.bool)
        if causal:
            see = torch.arange(n)[None] <= pos
            if window:
                see &= torch.arange(n)[None] > pos - window
        s = s.masked_fill(~see, -np.inf)
        w = torch.nan_to_num(torch.softmax(s, -1)) if n else s
        ref = torch.einsum("hij,jhd->ihd", w, v)
        np.testing.assert_allclose(out[rows], ref.numpy(), rtol=1e-12, atol=1e-12)
        z = torch.logsumexp(s, -1).T.numpy() if n else np.full((ql, Hq), -np.inf)
        np.testing.assert_allclose(lse[rows], z, rtol=1e-12)


def test_page_tables_by_hand():
    # page 4; ring of 6 with 3 free pages from entry 5 on: 50, 10, 11
    table = np.array([[7, -1, -1], [8, 9, -1], [3, -1, -1], [4, 5, -1], [6, -1, -1]], np.int32)
    ring = np.array([10, 11, -1, -1, -1, 50], np.int32)
    seq, start, slots, pos, state = kv_cache.page_tables(
        [3, 5, 4, 8, 2], [2, -1, 6, 1, 1], table, ring, [5, 3], 4, 12)
    # request 0 takes page 50; 1 gives 8 and 9 back; 2 takes 10 and 11; 3 finds none; 4 needs none
    assert seq.tolist() == [5, 0, 10, -1, 3] and start.tolist() == [0, 2, 2, 8, 9, 10]
    assert table[0].tolist() == [7, 50, -1] and table[2].tolist() == [3, 10, 11] and table[3].tolist() == [4, 5, -1]
    assert slots.tolist() == [31, 200, 40, 41, 42, 43, 44, 45, -1, 26, -1, -1]
    assert pos.tolist() == [3, 4, 4, 5, 6, 7, 8, 9, 8, 2, -1, -1]
    assert state.tolist() == [2, 2] and ring.tolist() == [10, 11, 8, 9, -1, 50]
