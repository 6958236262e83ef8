"""GPU parity of the 4-bit KV cache's tables, write and read-back with the
oracle: all of them exactly (page ids and slots are whole numbers, the
quantiser is a fixed rule, and a stored value is exact in bf16)."""

import numpy as np
import pytest
import torch

from oracle import kv_cache as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mxfp4_weight_only_gb300 import build

    build.build()
    import mxfp4_weight_only_gb300 as m

    return m


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ page tables


def tables_case(m, cached, new, mb, page, free, ring_size, head, max_tokens, seed=0):
    g = np.random.default_rng(seed)
    R = len(cached)
    have = [-(-c // page) for c in cached]
    ids = g.permutation(sum(have) + free + 5)
    table = g.integers(-1, 99, (R, mb)).astype(np.int32)
    at = 0
    for r in range(R):
        table[r, : have[r]] = ids[at: at + have[r]]
        at += have[r]
    ring = np.full(ring_size, -7, np.int32)
    ring[(head + np.arange(free)) % ring_size] = ids[at: at + free]
    want_table, want_ring = table.copy(), ring.copy()
    want = ref.page_tables(cached, new, want_table, want_ring, [head, free], page, max_tokens)
    bt, rg = i32(table), i32(ring)
    for _ in range(2):  # the same inputs again: the same tables again
        got = m.kv_page_tables(i32(cached), i32(new), bt, rg, i32([head, free]), page, max_tokens)
        for name, a, b in zip(got._fields, got, want):
            assert np.array_equal(a.cpu().numpy(), b), name
        assert np.array_equal(bt.cpu().numpy(), want_table) and np.array_equal(rg.cpu().numpy(), want_ring)


@pytest.mark.parametrize("R,page,lens,news,mb,free,max_tokens", [
    (1, 16, (0, 1), (1, 2), 1, 1, 1),             # the first token of the first request
    (1, 64, (0, 1), (0, 1), 2, 0, 5),             # nothing new
    (5, 16, (0, 40), (0, 40), 6, 40, 300),        # every request fits
    (40, 16, (0, 200), (0, 90), 20, 60, 4000),    # the pages run out
    (40, 32, (0, 200), (0, 90), 8, 200, 700),     # the tokens and the rows run out
    (700, 16, (0, 300), (1, 2), 40, 300, 1024),   # a decode step of many requests
    (1100, 128, (0, 900), (0, 60), 9, 900, 40001),
    (8192, 256, (0, 600), (0, 3), 4, 5000, 9000),
])
@pytest.mark.parametrize("release", [0.0, 0.3])
def test_page_tables(m, R, page, lens, news, mb, free, max_tokens, release):
    g = np.random.default_rng(R + page)
    new = g.integers(*news, R)
    new[g.random(R) < release] = -1
    cached = g.integers(*lens, R)
    ring_size = sum(-(-c // page) for c in cached) + free + 3
    tables_case(m, cached.tolist(), new.tolist(), mb, page, free, ring_size, ring_size - 2, max_tokens)


def test_page_tables_step_after_step(m):
    """Requests that grow, finish and start again on one ring never share a page."""
    g = np.random.default_rng(4)
    R, page, mb, C = 6, 16, 8, 30
    bt, ring = i32(np.full((R, mb), -1)), i32(np.arange(C))
    state, lens = i32([0, C]), np.zeros(R, np.int64)
    for step in range(30):
        new = g.integers(0, 40, R)
        new[g.random(R) < 0.25] = -1
        got = m.kv_page_tables(i32(lens), i32(new), bt, ring, state, page, 256)
        seq = got.seq_lens.cpu().numpy()
        lens = np.where(seq < 0, lens, seq)
        state = got.ring_state
        head, free = state.tolist()
        held = [bt.cpu().numpy()[r, b] for r in range(R) for b in range(-(-int(lens[r]) // page))]
        spare = ring.cpu().numpy()[(head + np.arange(free)) % C].tolist()
        assert sorted(held + spare) == list(range(C)), step


def test_page_tables_without_requests(m):
    got = m.kv_page_tables(i32([]), i32([]), i32(np.zeros((0, 4))), i32([3, 4]), i32([1, 2]), 16, 5)
    assert got.query_start.tolist() == [0] and got.slots.tolist() == [-1] * 5 and got.ring_state.tolist() == [1, 2]


# ------------------------------------------------------------------ write and read-back


def written(m, x, slots, heads, D, page, pages, seed=0, stream=None):
    """The cache's bytes before and after appending x = (k, v), and the cache."""
    before = torch.randint(0, 256, (pages, heads, page // 16, 17 * D), dtype=torch.uint8, device="cuda",
                           generator=torch.Generator("cuda").manual_seed(seed))
    c = m.KvCacheMxfp4(pages, page, heads, D, data=before.clone())
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    m.kv_append_mxfp4(c, x[0], x[1], i32(slots) if not torch.is_tensor(slots) else slots, stream=stream)
    if stream is not None:
        torch.cuda.current_stream().wait_stream(stream)
    return before.cpu().numpy(), c


def expect(before, x, slots, page, pages):
    data = before.copy()
    kc, ks = ref.quantize(x[0].float().cpu().numpy())
    vc, vs = ref.quantize(x[1].float().cpu().numpy())
    for i, s in enumerate(slots):
        if 0 <= s < pages * page:
            for h in range(data.shape[1]):
                ref.write(data, s, h, kc[i, h], ks[i, h], vc[i, h], vs[i, h])
    return data


def rows(n, heads, D, dtype, seed):
    g = np.random.default_rng(seed)
    x = g.standard_normal((2, n, heads, D)) * np.exp(2 * g.standard_normal((2, n, heads, 1)))
    return [torch.from_numpy(a).to("cuda", dtype) for a in x]


@pytest.mark.parametrize("n,heads,D,page,dtype", [
    (1, 1, 64, 16, torch.bfloat16), (1, 4, 128, 64, torch.bfloat16), (33, 3, 128, 16, torch.float32),
    (70, 5, 64, 32, torch.bfloat16), (17, 8, 128, 128, torch.bfloat16), (65, 2, 64, 256, torch.float32),
    (300, 1, 128, 16, torch.bfloat16),
])
def test_append_and_gather(m, n, heads, D, page, dtype):
    pages = -(-n // page) + 2
    x = rows(n, heads, D, dtype, n)
    slots = np.random.default_rng(n).permutation(pages * page)[:n]
    slots[n // 3:: 7] = -1
    before, c = written(m, x, slots, heads, D, page, pages)
    data = expect(before, x, slots, page, pages)
    assert np.array_equal(c.data.cpu().numpy(), data)  # every other byte is as it was
    k, v = m.kv_gather_mxfp4(c, i32(slots))
    live = slots >= 0
    kc, ks, vc, vs = ref.read(data, np.where(live, slots, 0))
    for got, codes, sc in ((k, kc, ks), (v, vc, vs)):
        want = np.where(live[:, None, None], ref.values(codes, sc), 0.0)
        assert np.array_equal(got.float().cpu().numpy(), want)


def test_append_prompt_in_order(m):
    """Consecutive slots over whole and partial groups of 16, from an offset in the page."""
    n, heads, D, page, pages = 213, 4, 128, 64, 5
    x = rows(n, heads, D, torch.bfloat16, 3)
    for off in (0, 5):
        t = np.arange(n) + off
        slots = np.array([3, 1, 4, 0, 2])[t // page] * page + t % page
        before, c = written(m, x, slots, heads, D, page, pages)
        assert np.array_equal(c.data.cpu().numpy(), expect(before, x, slots, page, pages))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_extreme_values(m, dtype):
    n, heads, D, page, pages = 64, 1, 128, 32, 2
    g = np.random.default_rng(8)
    x = g.standard_normal((2, n, heads, D)) * 2.0 ** g.integers(-140, 126, (2, n, heads, 1))
    x[0, 0] = 0.0
    x[0, 1] = -0.0
    x[1, 2, 0, 5] = np.nan
    x[1, 3, 0, [7, 40]] = np.inf, -np.inf
    x[0, 4, 0, 70], x[0, 4, 0, 71] = np.inf, np.nan
    x[0, 5, 0, :8] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]  # every tie
    x[0, 5, 0, 8:32] = 0
    x = [torch.from_numpy(a).to("cuda", dtype) for a in x]
    slots = g.permutation(n)
    before, c = written(m, x, slots, heads, D, page, pages)
    data = expect(before, x, slots, page, pages)
    assert np.array_equal(c.data.cpu().numpy(), data)
    k, v = m.kv_gather_mxfp4(c, i32(slots))
    kc, ks, vc, vs = ref.read(data, slots)
    for got, codes, sc in ((k, kc, ks), (v, vc, vs)):
        want = torch.from_numpy(ref.values(codes, sc)).to(torch.bfloat16).float().numpy()
        assert np.array_equal(got.float().cpu().numpy(), want, equal_nan=True)


def test_append_from_a_fused_projection_on_another_stream(m):
    n, heads, D, page, pages = 50, 2, 64, 16, 8
    x = rows(n, heads, D, torch.bfloat16, 5)
    qkv = torch.cat([torch.full((n, 640), 9.0, dtype=torch.bfloat16, device="cuda"), x[0].flatten(1), x[1].flatten(1)], 1)
    k = qkv[:, 640: 640 + heads * D].view(n, heads, D)
    v = qkv[:, 640 + heads * D:].view(n, heads, D)
    assert not k.is_contiguous()
    slots = np.random.default_rng(1).permutation(pages * page)[:n]
    before, c = written(m, (k, v), i32(slots), heads, D, page, pages, stream=torch.cuda.Stream())
    assert np.array_equal(c.data.cpu().numpy(), expect(before, x, slots, page, pages))


def test_slots_outside_the_cache_are_skipped(m):
    n, heads, D, page, pages = 6, 2, 64, 16, 3
    x = rows(n, heads, D, torch.bfloat16, 6)
    slots = np.array([-1, 48, 2 ** 31 - 1, -(2 ** 31), 47, 0])
    before, c = written(m, x, slots, heads, D, page, pages)
    assert np.array_equal(c.data.cpu().numpy(), expect(before, x, slots, page, pages))
    k, _ = m.kv_gather_mxfp4(c, i32(slots))
    assert (k[:4] == 0).all() and (k[4:] != 0).any()


def test_refusals(m):
    with pytest.raises(ValueError):
        m.KvCacheMxfp4(4, 24, 2, 64)
    with pytest.raises(ValueError):
        m.KvCacheMxfp4(4, 16, 2, 96)
    with pytest.raises(ValueError):
        m.KvCacheMxfp4(4, 16, 2, 64, data=torch.empty(4, 2, 1, 17 * 64, dtype=torch.uint8))
    c = m.KvCacheMxfp4(4, 16, 2, 64)
    x = rows(3, 2, 64, torch.bfloat16, 1)
    s = i32([0, 1, 2])
    with pytest.raises(TypeError):
        m.kv_append_mxfp4(c, x[0].half(), x[1].half(), s)
    with pytest.raises(TypeError):
        m.kv_append_mxfp4(c, x[0], x[1].float(), s)
    with pytest.raises(ValueError):
        m.kv_append_mxfp4(c, x[0][:2], x[1], s)
    with pytest.raises(ValueError):
        m.kv_append_mxfp4(c, x[0].transpose(0, 1).contiguous().transpose(0, 1), x[1], s)
    with pytest.raises(TypeError):
        m.kv_append_mxfp4(c, x[0], x[1], s.long())
    with pytest.raises(m.MoeError):  # rows not 16-byte aligned
        y = torch.zeros(3 * 128 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(3, 2, 64)
        m.kv_append_mxfp4(c, y, x[1], s)
    with pytest.raises(ValueError):
        m.kv_gather_mxfp4(c, s, k_out=torch.empty(3, 2, 128, dtype=torch.bfloat16, device="cuda"))
    t = [i32([1]), i32([1]), i32([[0, 1]]), i32([1, 2]), i32([0, 2])]
    with pytest.raises(ValueError):
        m.kv_page_tables(*t, 16, 4, ring_state_out=t[4])
    with pytest.raises(ValueError):
        m.kv_page_tables(t[0], i32([1, 2]), *t[2:], 16, 4)
    with pytest.raises(m.MoeError):
        m.kv_page_tables(*t, 20, 4)
    torch.cuda.synchronize()
