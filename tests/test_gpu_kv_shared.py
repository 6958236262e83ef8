"""GPU parity of attention behind a shared prefix with the float64 oracle.

The bound is that of attention over the cache, from the arithmetic alone: the result
is rounded to bf16 (2^-8 of it); each weight p_j enters its product rounded to f16 or bf16
(2^-9 of sum p|v|, the oracle's ``spread``); a score is a float32 sum of D
products, off by at most D 2^-24 of sum |scale q_d k_d| (``size``), and moves
its weight by twice that share of ``spread``; the exponentials and sums add a
few 2^-22, covered by 2^-13, the joining of the parts among them: each is weighted by one
more exponential, of a difference of references that is off by 2^-24 of the larger, which
is at most ``size`` times log2 e.
    |out - ref| <= (2^-8 + 2^-13) |ref| + (2^-9 + 2^-13 + 2 (D + 2) 2^-24 size) spread
    |lse - ref| <= (D + 2) 2^-24 size + 2^-20 (1 + |ref|)
On top comes what weights below 2^-126 of the largest add, which float32 exponentials lose:
at most 2^-126 (keys) max |v|, max |v| being 6 2^(s - 127) for the largest value scale s.
(Found by keys that hold a dimension's only value 2^138 below the heaviest key, with
values of 2^16: 2.6e-37, where the float32 weight is 0.)
Where a part has more than 256 keys, the tensor-core kernel holds its weights p 2^9 in f16, 11 bits down to
p = 2^-23 of the part's reference and multiples of 2^-33 below, off by at most 2^-34: as in the tests
of prompts without a prefix, 2^-34 of sum |v|, at most 2^-34 (keys) max |v|, comes on top there.  (The reference is
a score of the part, so that its sum of weights is at least 1, and a part enters the result with a weight of at
most 1.  Found by a dimension whose heaviest key has the value 0: 1.8e-8, 2.1e-10 off.)
Results near or below the smallest normal number are held to 1e-37, eight times its size (as there).
Rows outside every request are not written.
"""

import numpy as np
import pytest
import torch

from oracle import kv_shared as ref

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


def problem(P, lens, qlens, H, G, D, page, seed=0, bands=((120, 127), (120, 127)), extra=1, gaps=0):
    """Random codes, scale bytes in ``bands`` (K, V); everything past a length is garbage."""
    g = np.random.default_rng(seed + P)
    R = len(lens)
    need = [-(-max(n, 0) // page) for n in lens]
    first = -(-P // page)
    mb, sb = max([1] + need) + extra, max(1, first + extra)
    pages = first + sum(need) + 2
    ids = g.permutation(pages).tolist()
    data = g.integers(0, 256, (pages, H, page // 16, 17 * D), dtype=np.uint8)
    table = g.integers(-5, pages + 5, (R, mb)).astype(np.int32)
    shared = g.integers(-5, pages + 5, sb).astype(np.int32)
    NB = D // 32

    def live(page_id, j):
        rec = data[page_id, :, j % page // 16]
        for w in range(2):
            at = 16 * D + w * (D // 2) + j % 16 * NB
            rec[:, at: at + NB] = g.integers(bands[w][0], bands[w][1] + 1, (H, NB))

    for b in range(first):
        shared[b] = ids.pop()
    for j in range(P):
        live(shared[j // page], j)
    for r, n in enumerate(lens):
        for b in range(need[r]):
            table[r, b] = ids.pop()
        for j in range(max(n, 0)):
            live(table[r, j // page], j)
    start = np.concatenate([[0], np.cumsum(qlens)])
    q = torch.from_numpy(g.standard_normal((start[-1] + gaps, H * G, D))).to(torch.bfloat16)
    return dict(q=q, data=data, shared=shared, P=P, table=table, lens=np.array(lens), start=start, H=H, G=G, D=D, page=page, pages=pages,
                lost=(2.0 ** -126 + (2.0 ** -34 if max(P, *lens) > 256 else 0)) * (P + max(lens)) * 6 * 2.0 ** (bands[1][1] - 127))


def run(m, p, scale=0.2, causal=True, q=None, stream=None, max_q=None):
    c = m.KvCacheMxfp4(p["pages"], p["page"], p["H"], p["D"], data=torch.from_numpy(p["data"]).cuda())
    q = p["q"].cuda() if q is None else q
    N, Hq, D = q.shape
    out = torch.full((N, Hq, D), 77.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((N, Hq), 77.0, device="cuda")
    if max_q is None:
        max_q = int(np.diff(p["start"]).max())
    n = m.attention_shared_workspace_bytes(c, len(p["lens"]), N, Hq, p["table"].shape[1], max_q, len(p["shared"]))
    ws = torch.randint(0, 256, (n,), dtype=torch.uint8, device="cuda")  # contents do not matter
    ws[:4] = 0
    args = (q, c, i32(p["shared"]), i32([p["P"]]), i32(p["table"]), i32(p["lens"]), i32(p["start"]), max_q)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    got = m.attention_kv_mxfp4_shared(*args, scale=scale, causal=causal, out=out, lse=lse, workspace=ws, stream=stream)
    assert got is out
    if stream is not None:
        torch.cuda.current_stream().wait_stream(stream)
    assert m.attention_read_status(ws) == 0
    return out, lse


def check(p, out, lse, scale=0.2, causal=True):
    want, wl, spread, size = ref.attention(p["q"].float().numpy(), p["data"], p["shared"], p["P"], p["table"], p["lens"],
                                           p["start"], scale, causal)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    n = p["start"][-1]
    assert (got[n:] == 77.0).all() and (gl[n:] == 77.0).all()
    got, gl, want, wl, spread, size = (x[:n] for x in (got, gl, want, wl, spread, size))
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isnan(gl), np.isnan(wl))
    sum_err = (p["D"] + 2) * 2.0 ** -24 * size
    bound = (2.0 ** -8 + 2.0 ** -13) * np.abs(want) + (2.0 ** -9 + 2.0 ** -13 + 2 * sum_err[..., None]) * spread
    with np.errstate(invalid="ignore"):
        bad = np.abs(got - want) > bound + p["lost"] + 1e-37
        off = np.abs(gl - wl) > sum_err + 2.0 ** -20 * (1 + np.abs(wl))
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], bound[bad][:4])
    empty = np.isinf(wl)
    assert np.array_equal(gl[empty], wl[empty])
    assert not (off & ~empty).any(), (np.argwhere(off & ~empty)[:4], gl[off & ~empty][:4], wl[off & ~empty][:4])


def both(m, p, scale=0.2, **kw):
    out, lse = run(m, p, scale, **kw)
    check(p, out, lse, scale, kw.get("causal", True))


@pytest.mark.parametrize("H,G,D", [(1, 1, 64), (4, 7, 128), (2, 8, 128), (3, 5, 64), (1, 64, 128), (8, 1, 128)])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("P", [0, 1, 15, 16, 17, 127, 128, 129, 300])
def test_decode(m, H, G, D, page, P):
    both(m, problem(P, [1, 0, 15, -1, 16, 100], [1] * 6, H, G, D, page, seed=H * G))


@pytest.mark.parametrize("R", [1, 2, 8, 9, 33, 70])
@pytest.mark.parametrize("P", [500, 2100])
def test_batches(m, R, P):
    g = np.random.default_rng(R)
    both(m, problem(P, g.integers(1, 40, R).tolist(), [1] * R, 2, 4, 64, 32, seed=R))


@pytest.mark.parametrize("G,D,q", [(1, 64, 4), (7, 128, 2), (4, 64, 40), (2, 128, 129), (16, 64, 5)])
@pytest.mark.parametrize("causal", [True, False])
def test_several_query_rows(m, G, D, q, causal):
    lens = [max(0, q - 2), q, q + 1, q + 150, -1, 17 + q]
    both(m, problem(700, lens, [q, q, q, q, 3, max(1, q // 2)], 2, G, D, 32, seed=q, gaps=3), causal=causal)


@pytest.mark.parametrize("G,D,lens,qlens", [
    (7, 128, [300, 1, 200], [300, 1, 123]), (1, 64, [257, 1500], [257, 1300]), (16, 64, [130, 64, -1, 90], [130, 64, 2, 1]),
    (5, 128, [500, 0, 129], [370, 30, 128]),
])
@pytest.mark.parametrize("causal", [True, False])
def test_prompts_behind_a_prefix(m, G, D, lens, qlens, causal):
    """Enough rows a request for the tensor-core kernel on its own keys too."""
    both(m, problem(333, lens, qlens, 2, G, D, 64, seed=len(lens) + G), causal=causal, scale=0.1)


def test_many_requests(m):
    g = np.random.default_rng(2)
    both(m, problem(200, g.integers(-1, 30, 700).tolist(), [1] * 700, 1, 2, 64, 16))


def test_workspace_of_a_larger_batch(m):
    """Fewer rows can be cut into more slices: a workspace for more of them has to do."""
    H, G, D = 4, 7, 128
    c = m.KvCacheMxfp4(4, 16, H, D)
    size = [m.attention_shared_workspace_bytes(c, R, R, H * G, 1, 1, 512) for R in range(1, 80)]
    R = next(i for i, (a, b) in enumerate(zip(size, size[1:]), 1) if a > b)
    p = problem(512 * 16 - 3, [10] * R, [1] * R, H, G, D, 16, seed=3, extra=0)
    assert len(p["shared"]) == 512 and p["table"].shape[1] == 1
    c = m.KvCacheMxfp4(p["pages"], 16, H, D, data=torch.from_numpy(p["data"]).cuda())
    q = p["q"].cuda()
    out, lse = torch.empty_like(q), torch.empty(R, H * G, device="cuda")
    args = (q, c, i32(p["shared"]), i32([p["P"]]), i32(p["table"]), i32(p["lens"]), i32(p["start"]), 1)
    ws = torch.zeros(m.attention_shared_workspace_bytes(c, R + 1, R + 1, H * G, 1, 1, 512), dtype=torch.uint8, device="cuda")
    m.attention_kv_mxfp4_shared(*args, scale=0.2, out=out, lse=lse, workspace=ws)
    check(p, out, lse)
    with pytest.raises(m.MoeError, match="WORKSPACE"):
        m.attention_kv_mxfp4_shared(*args, scale=0.2, out=out, lse=lse, workspace=ws[: ws.numel() // 32])


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_page_sizes(m, page):
    both(m, problem(777, [5, 257, 40] * 4, [1] * 12, 2, 4, 128, page, seed=page))


def test_long_prefix_is_cut(m):
    both(m, problem(20011, [30] * 12, [1] * 12, 1, 8, 128, 128), scale=0.05)  # tensor cores, many slices
    both(m, problem(20011, [30, 1], [1, 1], 1, 8, 64, 16), scale=0.05)  # streamed


def test_shorter_than_its_table(m):
    """The plan is made for the table's pages, the length may be anything below."""
    for n in (1, 130, 1000, 4000):
        p = problem(4096, [20] * 10, [1] * 10, 2, 4, 64, 64, seed=n)
        p["P"] = n
        both(m, p)
    p["P"] = -3
    out, lse = run(m, p)
    p["P"] = 0
    check(p, out, lse)
    p["P"] = 2 ** 31 - 1  # more than the table holds: what its pages are
    p["shared"][-1] = 99999
    out, lse = run(m, p)
    p["P"] = 64 * len(p["shared"])
    check(p, out, lse)


def test_nothing_to_see(m):
    p = problem(0, [0, -1, 3, 0], [2, 1, 1, 20], 2, 4, 64, 16)
    both(m, p)
    p = problem(100, [-1] * 12, [1] * 12, 2, 4, 64, 16)
    out, lse = run(m, p)
    assert (out == 0).all() and torch.isinf(lse).all()


def test_bad_pages_are_invisible(m):
    p = problem(900, [50] * 12, [1] * 12, 2, 4, 128, 16, seed=5)
    p["shared"][[0, 7, 30, 55]] = [-1, 10 ** 6, p["pages"], -2 ** 31]
    p["table"][3, 1] = -1
    p["table"][4, :] = 2 ** 31 - 1
    both(m, p)
    p["shared"][:] = -1
    both(m, p)


@pytest.mark.parametrize("R", [3, 20])
@pytest.mark.parametrize("bands", [((0, 60), (120, 127)), ((120, 127), (0, 90)), ((60, 150), (100, 200)), ((150, 158), (140, 240)),
                                   ((104, 104), (0, 0)), ((140, 141), (140, 141))])
def test_scales_of_any_size(m, R, bands):
    both(m, problem(600, [40] * R, [1] * R, 2, 4, 64, 32, seed=R, bands=bands), scale=0.01)


@pytest.mark.parametrize("R", [3, 20])
def test_nan_tokens(m, R):
    p = problem(500, [40] * R, [1] * R, 2, 4, 64, 32, seed=1)
    NB = 2
    def poison(page_id, j, head, w, s=255):  # noqa: E306
        p["data"][page_id, head, j % 32 // 16, 16 * 64 + w * 32 + j % 16 * NB] = s
    poison(p["table"][1, 0], 5, 0, 0)
    poison(p["table"][2, 1], 36, 1, 1)
    both(m, p)
    poison(p["shared"][100 // 32], 100, 1, 0)  # everybody sees the prefix's token of head 1
    out, lse = run(m, p)
    check(p, out, lse)
    assert torch.isnan(lse[0, 4:]).all() and torch.isfinite(lse[0, :4]).all()


@pytest.mark.parametrize("R", [2, 20])
def test_not_finite_queries(m, R):
    p = problem(300, [10] * R, [1] * R, 2, 4, 64, 32, seed=2)
    p["q"][1, 3, 7] = float("inf")
    out, lse = run(m, p)
    assert torch.isnan(out[1, 3].float()).all() and torch.isnan(lse[1, 3])
    p["q"][1, 3, 7] = 0.0
    want = run(m, p)
    keep = torch.ones(R, 8, dtype=torch.bool, device="cuda")
    keep[1, 3] = False
    assert torch.allclose(out[keep].float(), want[0][keep].float(), rtol=2 ** -6, atol=2 ** -7)
    check(p, *want)


@pytest.mark.parametrize("R", [2, 20])
@pytest.mark.parametrize("where", ["prefix", "own"])
def test_huge_scores(m, R, where):
    """Scores of 2^30 in one of the parts: the other's weigh nothing, ties within a part hold."""
    p = problem(260, [40] * R, [1] * R, 1, 4, 64, 32, seed=3, bands=((127, 127), (127, 127)))
    NB = 2
    pages = [p["shared"]] if where == "prefix" else list(p["table"])
    for t in pages:
        for j in (3, 21):
            p["data"][t[0], 0, j // 16, 16 * 64 + j % 16 * NB: 16 * 64 + (j % 16 + 1) * NB] = 157
    out, lse = run(m, p, scale=1.0)
    check(p, out, lse, 1.0)


def test_equal_scores_across_the_parts(m):
    """All scores are 0: the plain mean over the prefix's and own values."""
    p = problem(1000, [24] * 12, [1] * 12, 2, 4, 128, 16, seed=4)
    p["q"].zero_()
    both(m, p)


def test_negative_and_zero_scale(m):
    p = problem(400, [24] * 12, [1] * 12, 2, 4, 128, 16, seed=6)
    both(m, p, scale=-0.15)
    both(m, p, scale=0.0)


def test_strided_queries_and_other_stream(m):
    p = problem(400, [24] * 12, [1] * 12, 2, 4, 128, 16, seed=7)
    wide = torch.full((12, 14, 128), 1e30, dtype=torch.bfloat16, device="cuda")
    wide[:, :8] = p["q"].cuda()
    both(m, p, q=wide[:, :8], stream=torch.cuda.Stream())


def test_rows_cut_by_max_q_len(m):
    p = problem(200, [30, 30, 30], [9, 9, 9], 2, 4, 64, 16, seed=8)
    out, lse = run(m, p, max_q=4)
    want, _ = run(m, p)
    for r in range(3):
        assert torch.equal(out[9 * r: 9 * r + 4], want[9 * r: 9 * r + 4])
        assert (out[9 * r + 4: 9 * r + 9] == 77.0).all() and (lse[9 * r + 4: 9 * r + 9] == 77.0).all()


def test_same_as_without_a_prefix(m):
    """Against attention over one table that holds both (a prefix of whole pages)."""
    p = problem(640, [33] * 16, [1] * 16, 2, 7, 128, 32, seed=9, extra=0)
    c = m.KvCacheMxfp4(p["pages"], 32, 2, 128, data=torch.from_numpy(p["data"]).cuda())
    both_tables = np.concatenate([np.tile(p["shared"], (16, 1)), p["table"]], 1)
    lse = torch.empty(16, 14, device="cuda")
    want = m.attention_kv_mxfp4(p["q"].cuda(), c, i32(both_tables), i32(p["lens"] + 640), i32(p["start"]), 1, scale=0.2, lse=lse)
    out, got = run(m, p)
    assert torch.allclose(out.float(), want.float(), rtol=2 ** -6, atol=2 ** -8) and torch.allclose(got, lse, atol=1e-4)


@pytest.mark.parametrize("R", [2, 30])
def test_captured_and_repeatable(m, R):
    p = problem(1500, [20] * R, [1] * R, 2, 7, 128, 64, seed=10)
    c = m.KvCacheMxfp4(p["pages"], 64, 2, 128, data=torch.from_numpy(p["data"]).cuda())
    q, P, lens = p["q"].cuda(), i32([100]), i32([3] * R)
    shared, table, start = i32(p["shared"]), i32(p["table"]), i32(p["start"])
    ws = torch.zeros(m.attention_shared_workspace_bytes(c, R, R, 14, table.shape[1], 1, len(shared)), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(R, 14, device="cuda")

    def call():
        m.attention_kv_mxfp4_shared(q, c, shared, P, table, lens, start, 1, scale=0.2, out=out, lse=lse, workspace=ws)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    P.fill_(1500)
    lens.fill_(20)
    graph.replay()
    check(p, out, lse)
    first = out.clone()
    for _ in range(3):
        graph.replay()
        assert torch.equal(out, first)


def test_refusals(m):
    p = problem(40, [5, 6], [1, 1], 2, 4, 64, 16)
    c = m.KvCacheMxfp4(p["pages"], 16, 2, 64, data=torch.from_numpy(p["data"]).cuda())
    q = p["q"].cuda()
    ok = dict(shared_table=i32(p["shared"]), shared_len=i32([40]), block_table=i32(p["table"]), seq_lens=i32(p["lens"]),
              query_start=i32(p["start"]), max_q_len=1)
    for kw, e in ((dict(shared_len=i32([40, 1])), ValueError), (dict(shared_len=torch.tensor([40], device="cuda")), TypeError),
                  (dict(shared_table=i32(p["table"])), ValueError), (dict(shared_table=i32([])), m.MoeError),
                  (dict(max_q_len=-1), m.MoeError), (dict(scale=float("nan")), m.MoeError), (dict(out=q), m.MoeError),
                  (dict(workspace=torch.zeros(4096, dtype=torch.uint8, device="cuda")), m.MoeError),
                  (dict(shared_table=i32(p["shared"]).cpu()), ValueError)):
        with pytest.raises(e):
            m.attention_kv_mxfp4_shared(q, c, **{**ok, **kw})
    with pytest.raises(TypeError):
        m.attention_kv_mxfp4_shared(q.float(), c, **ok)
    m.attention_kv_mxfp4_shared(q, c, **ok)
    torch.cuda.synchronize()
