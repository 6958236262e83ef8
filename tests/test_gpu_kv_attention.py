"""GPU parity of attention over the 4-bit cache with the float64 oracle.

Bound per output element, from the arithmetic alone: the result is rounded to
bf16 (2^-9 of it); each weight p_j enters its product rounded to f16 or bf16
(2^-9 of sum p|v|, the oracle's ``spread``); a score is a float32 sum of D
products, off by at most D 2^-24 of sum |scale q_d k_d| (``size``), and moves
its weight by twice that share of ``spread``; the exponentials and sums add a
few 2^-22, covered by 2^-13.
    |out - ref| <= (2^-9 + 2^-13) |ref| + (2^-9 + 2^-13 + 2 D 2^-24 size) spread
    |lse - ref| <= D 2^-24 size + 2^-20 (1 + |ref|)
Rows outside every request are not written.
"""

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


def problem(lens, qlens, H, G, D, page, seed=0, bands=((120, 127), (120, 127)), extra_blocks=1, gaps=0):
    """Random codes, scale bytes in ``bands`` (K, V); everything past a request's length is garbage."""
    g = np.random.default_rng(seed)
    R = len(lens)
    mb = max(1, max(-(-n // page) for n in lens)) + extra_blocks
    pages = sum(-(-n // page) for n in lens) + 2
    ids = g.permutation(pages).tolist()
    data = g.integers(0, 256, (pages, H, page // 16, 17 * D), dtype=np.uint8)
    table = g.integers(-5, pages + 5, (R, mb)).astype(np.int32)
    NB = D // 32
    for r, n in enumerate(lens):
        for b in range(-(-n // page)):
            table[r, b] = ids.pop()
        for j in range(n):
            rec = data[table[r, j // page], :, j % page // 16]
            for w in range(2):
                at = 16 * D + w * (D // 2) + j % 16 * NB
                rec[:, at: at + NB] = g.integers(bands[w][0], bands[w][1] + 1, (H, NB))
    start = np.concatenate([[0], np.cumsum(qlens)])
    q = g.standard_normal((start[-1] + gaps, H * G, D))
    q = torch.from_numpy(q).to(torch.bfloat16)
    return dict(q=q, data=data, table=table, lens=np.array(lens), start=start, H=H, G=G, D=D, page=page, pages=pages)


def run(m, p, scale, causal=True, window=0, q=None, stream=None, max_q=None, workspace=None):
    c = m.KvCacheMxfp4(p["pages"], p["page"], p["H"], p["D"], data=torch.from_numpy(p["data"]).cuda())
    q = p["q"].cuda() if q is None else q
    N, Hq, D = q.shape
    out = torch.full((N, Hq, D), 77.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((N, Hq), 77.0, device="cuda")
    if max_q is None:
        max_q = int(np.diff(p["start"]).max()) if len(p["lens"]) else 0
    args = (i32(p["table"]), i32(p["lens"]), i32(p["start"]))
    if workspace is None:
        n = m.attention_workspace_bytes(c, len(p["lens"]), N, Hq, p["table"].shape[1], max_q)
        workspace = torch.randint(0, 256, (n,), dtype=torch.uint8, device="cuda")  # contents do not matter
        workspace[:4] = 0
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    m.attention_kv_mxfp4(q, c, *args, max_q, scale=scale, causal=causal, window=window, out=out, lse=lse,
                         workspace=workspace, stream=stream)
    if stream is not None:
        torch.cuda.current_stream().wait_stream(stream)
    assert m.attention_read_status(workspace) == 0
    return out, lse


def check(p, out, lse, scale, causal=True, window=0):
    want, wl, spread, size = ref.attention(p["q"].float().numpy(), p["data"], p["table"], p["lens"], p["start"], scale,
                                           causal, window)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    n = p["start"][-1]
    assert (got[n:] == 77.0).all() and (gl[n:] == 77.0).all()
    got, gl, want, wl, spread, size = (x[:n] for x in (got, gl, want, wl, spread, size))
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isnan(gl), np.isnan(wl))
    D = p["D"]
    sum_err = D * 2.0 ** -24 * size
    bound = (2.0 ** -9 + 2.0 ** -13) * np.abs(want) + (2.0 ** -9 + 2.0 ** -13 + 2 * sum_err[..., None]) * spread
    with np.errstate(invalid="ignore"):
        bad = np.abs(got - want) > bound + 1e-37
        off = np.abs(gl - wl) > sum_err + 2.0 ** -20 * (1 + np.abs(wl))
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], bound[bad][:4])
    empty = np.isinf(wl)
    assert np.array_equal(gl[empty], wl[empty])
    assert not (off & ~empty).any(), (np.argwhere(off & ~empty)[:4], gl[off & ~empty][:4], wl[off & ~empty][:4])


def both(m, p, scale=0.2, **kw):
    out, lse = run(m, p, scale, **kw)
    check(p, out, lse, scale, kw.get("causal", True), kw.get("window", 0))


@pytest.mark.parametrize("H,G,D", [(1, 1, 64), (4, 7, 128), (2, 8, 128), (3, 5, 64), (1, 16, 128), (2, 12, 64), (1, 64, 128),
                                   (1, 33, 64), (8, 1, 128)])
@pytest.mark.parametrize("page", [16, 64])
def test_decode(m, H, G, D, page):
    both(m, problem([1, 0, 15, 16, 17, 100, 333, 1000], [1] * 8, H, G, D, page, seed=H * G))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_page_sizes(m, page):
    both(m, problem([5, 257, 600], [1, 1, 1], 2, 4, 128, page, seed=page))


def test_long_context_is_split(m):
    both(m, problem([20011], [1], 1, 8, 128, 128), scale=0.05)
    both(m, problem([9000, 3], [1, 1], 2, 3, 64, 16), scale=0.05)


def test_many_requests(m):
    g = np.random.default_rng(2)
    n = g.integers(0, 90, 700)
    both(m, problem(n.tolist(), [1] * 700, 1, 2, 64, 16))


@pytest.mark.parametrize("G,D,q", [(1, 64, 4), (7, 128, 2), (8, 128, 3), (16, 64, 5), (3, 128, 9), (4, 64, 40),
                                   (2, 128, 129)])
@pytest.mark.parametrize("window", [0, 1, 20, 200])
def test_several_query_rows(m, G, D, q, window):
    # contexts shorter than, equal to and longer than the rows; the first leaves rows empty
    lens = [max(0, q - 2), q, q + 1, q + 150, 17 + q]
    both(m, problem(lens, [q, q, q, q, max(1, q // 2)], 2, G, D, 32, seed=q, gaps=3), window=window)


@pytest.mark.parametrize("G,D,lens,qlens", [
    (7, 128, [300, 1, 700], [300, 1, 123]), (1, 64, [257, 400], [257, 300]), (4, 128, [1000], [1000]),
    (16, 64, [130, 64, 90], [130, 64, 1]), (5, 128, [2000, 50, 129], [70, 50, 128]),
])
@pytest.mark.parametrize("causal", [True, False])
def test_prompts(m, G, D, lens, qlens, causal):
    both(m, problem(lens, qlens, 2, G, D, 64, seed=len(lens) + G), causal=causal, scale=0.1)


@pytest.mark.parametrize("window", [1, 64, 129, 500])
def test_prompt_window(m, window):
    both(m, problem([700, 300], [600, 300], 1, 4, 128, 64), window=window)


def test_rows_of_no_request_and_empty_requests(m):
    p = problem([0, 40, 0, 0, 9], [0, 1, 0, 1, 1], 2, 4, 64, 16, gaps=2)
    both(m, p)
    p = problem([0, 0], [3, 200], 2, 4, 128, 16)
    both(m, p)
    p["lens"] = np.array([-1, -5])
    both(m, p)


def test_invalid_pages_hide_their_tokens(m):
    for qlens in ([1, 1], [90, 120]):
        p = problem([200, 150], qlens, 2, 4, 128, 16, seed=5)
        p["table"][0, [0, 3]] = -1, p["pages"]
        p["table"][1, 9] = 2 ** 31 - 1
        both(m, p)
        p["table"][1, :] = -9
        both(m, p)


def test_lengths_beyond_the_table_are_cut(m):
    p = problem([100, 64], [1, 1], 1, 4, 64, 16, extra_blocks=0)
    p["lens"] = np.array([10 ** 9, 64])
    p["table"][:, -1] %= p["pages"]
    p["data"][..., 16 * 64:] = 124
    both(m, p)


@pytest.mark.parametrize("qlen", [1, 100])
def test_not_a_number(m, qlen):
    p = problem([130, 130, 130], [qlen] * 3, 2, 4, 128, 16, seed=6)
    D, NB = 128, 4
    p["data"][p["table"][0, 2], 0, 0, 16 * D + 5 * NB + 1] = 255          # a key of request 0, head 0
    p["data"][p["table"][1, 7], 1, 0, 16 * D + D // 2 + 9 * NB] = 255     # a value of request 1, head 1
    p["data"][p["table"][2, 8], 0, 0, 16 * D + 1 * NB] = 255              # the last key of request 2
    both(m, p)
    both(m, p, window=3)


@pytest.mark.parametrize("qlen", [1, 60])
@pytest.mark.parametrize("bands,scale", [
    (((100, 150), (100, 150)), 2e-8),  # wide scales
    (((127, 128), (0, 254)), 0.1),     # values over the whole range of E8M0 (below infinity by the codes' 6)
    (((0, 3), (0, 3)), 1.0),           # nearly nothing
    (((117, 122), (245, 251)), 0.5),   # huge values
    (((230, 250), (124, 127)), 1e-33), # huge keys
    (((127, 129), (127, 127)), 3.0),   # sharp weights
])
def test_scales_of_any_size(m, qlen, bands, scale):
    p = problem([70, 200, 33], [qlen] * 2 + [1], 1, 4, 128, 16, seed=7, bands=bands)
    if bands[1] == (0, 254):
        # weights of very unlike size: tokens of few classes, so that small values count too
        v = p["data"].reshape(-1, 17 * 128)[:, 16 * 128 + 64:].view()
        v[v > 251] = 251
    both(m, p, scale=scale)


def test_dominant_key_with_small_values(m):
    """The key with nearly all the weight has values 2^60 times smaller than the others'."""
    p = problem([64], [1], 1, 4, 128, 16, seed=9)
    D, NB = 128, 4
    q = np.ones((1, 4, D))
    p["q"] = torch.from_numpy(q).to(torch.bfloat16)
    for j in range(64):
        rec = p["data"][p["table"][0, j // 16], 0, 0]
        for b in range(D // 2):
            rec[ref.k_at(j % 16, b, D)] = 0x77 if j == 21 else 0xFF
        rec[16 * D + j % 16 * NB: 16 * D + (j % 16 + 1) * NB] = 127
        rec[16 * D + D // 2 + j % 16 * NB: 16 * D + D // 2 + (j % 16 + 1) * NB] = 60 if j == 21 else 120
    both(m, p, scale=0.05)  # scores +-38: the others weigh e^-77


def test_strided_queries_on_another_stream(m):
    p = problem([90, 40, 300], [1, 1, 70], 2, 4, 128, 16, seed=3)
    N, Hq, D = p["q"].shape
    wide = torch.full((N, Hq * D + 512), 5.0, dtype=torch.bfloat16, device="cuda")
    wide[:, : Hq * D] = p["q"].cuda().flatten(1)
    q = wide[:, : Hq * D].view(N, Hq, D)
    out, lse = run(m, p, 0.2, q=q, stream=torch.cuda.Stream())
    check(p, out, lse, 0.2)


def test_repeated_calls_agree_bit_for_bit(m):
    p = problem([3000, 17, 900], [1, 1, 200], 2, 7, 128, 64, seed=11)
    a = run(m, p, 0.1)
    for _ in range(3):
        b = run(m, p, 0.1)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_one_workspace_for_calls_of_other_sizes(m):
    big = problem([3000, 17, 900], [1, 90, 200], 2, 7, 128, 64, seed=12)
    small = problem([40, 500], [1, 1], 2, 7, 128, 64, seed=13)
    c = m.KvCacheMxfp4(1, 64, 2, 128)
    ws = torch.zeros(max(m.attention_workspace_bytes(c, 3, 291, 14, big["table"].shape[1], 200),
                         m.attention_workspace_bytes(c, 2, 2, 14, small["table"].shape[1], 1)), dtype=torch.uint8, device="cuda")
    for p in (big, small, big, small):
        out, lse = run(m, p, 0.1, workspace=ws)
        check(p, out, lse, 0.1)


def test_captured_in_a_graph(m):
    p = problem([300, 5, 2000], [1, 1, 1], 2, 4, 128, 64, seed=14)
    c = m.KvCacheMxfp4(p["pages"], 64, 2, 128, data=torch.from_numpy(p["data"]).cuda())
    q, args = p["q"].cuda(), [i32(p["table"]), i32(p["lens"]), i32(p["start"])]
    ws = torch.zeros(m.attention_workspace_bytes(c, 3, 3, 8, p["table"].shape[1], 1), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(3, 8, device="cuda")
    call = lambda: m.attention_kv_mxfp4(q, c, *args, 1, scale=0.1, out=out, lse=lse, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    args[1].copy_(i32([128, 0, 1999]))  # the lengths are read when the graph runs
    g.replay()
    torch.cuda.synchronize()
    p["lens"] = np.array([128, 0, 1999])
    check(p, out, lse, 0.1)


def test_offsets_beyond_32_bits(m):
    """Pages past byte 2^32 of the cache (4.9 GB)."""
    H, D, page, pages = 8, 128, 64, 70000
    data = torch.empty((pages, H, page // 16, 17 * D), dtype=torch.uint8, device="cuda")
    p = problem([150, 90], [1, 70], H, 2, D, page, seed=15)
    far = np.arange(p["pages"]) + pages - p["pages"]
    data[far[0]:] = torch.from_numpy(p["data"]).cuda()
    ok = (p["table"] >= 0) & (p["table"] < p["pages"])
    table = np.where(ok, p["table"] + far[0], -1)
    c = m.KvCacheMxfp4(pages, page, H, D, data=data)
    q = p["q"].cuda()
    lse = torch.empty(q.shape[:2], device="cuda")
    out = m.attention_kv_mxfp4(q, c, i32(table), i32(p["lens"]), i32(p["start"]), 70, scale=0.1, lse=lse)
    check(p, out, lse, 0.1)
    # the write and the read-back at the last slots
    x = torch.randn(2, 3, H, D, device="cuda").bfloat16()
    s = i32([pages * page - 1, pages * page - 17, pages * page - 33])
    m.kv_append_mxfp4(c, x[0], x[1], s)
    k, v = m.kv_gather_mxfp4(c, s)
    for got, want in ((k, x[0]), (v, x[1])):
        codes = ref.quantize(want.float().cpu().numpy())
        assert np.array_equal(got.float().cpu().numpy(), ref.values(*codes))


def test_refusals(m):
    p = problem([40], [1], 2, 4, 64, 16)
    c = m.KvCacheMxfp4(p["pages"], 16, 2, 64)
    q, t, n, s = p["q"].cuda(), i32(p["table"]), i32([40]), i32([0, 1])
    ok = lambda **kw: m.attention_kv_mxfp4(kw.pop("q", q), c, kw.pop("t", t), kw.pop("n", n), kw.pop("s", s), 1, **kw)  # noqa: E731
    ok()
    for kw, err in ((dict(q=q.float()), TypeError), (dict(q=q[..., :32]), ValueError), (dict(q=q.cpu()), ValueError),
                    (dict(q=q[:, :7].contiguous()), m.MoeError), (dict(t=t.long()), TypeError), (dict(t=t[0]), ValueError),
                    (dict(s=i32([0])), ValueError), (dict(window=-1), m.MoeError), (dict(window=3, causal=False), m.MoeError),
                    (dict(scale=float("nan")), m.MoeError), (dict(out=torch.empty_like(q[..., :32])), ValueError),
                    (dict(lse=torch.empty(1, 4, device="cuda")), ValueError),
                    (dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")), m.MoeError)):
        with pytest.raises(err):
            ok(**kw)
    torch.cuda.synchronize()
