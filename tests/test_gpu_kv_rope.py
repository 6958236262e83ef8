"""GPU parity of the rotating cache write with the oracle, exactly: the rotation's
products and sums are rounded one by one, the quantiser is a fixed rule, and the
queries' rounding to bf16 is one more."""

import numpy as np
import pytest
import torch

from oracle import block, kv_cache as ref

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


def table(n, rot, base=10000.0):
    a = np.arange(n)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def case(m, N, Hq, H, D, rot, page=16, f32=False, pairs=False, seed=0, offset=0, far=700, strided=False, edit=None, stream=None):
    g = np.random.default_rng(seed + N + Hq + rot)
    pages = -(-N // page) + 2
    dt = torch.float32 if f32 else torch.bfloat16
    ch = np.exp(g.standard_normal(D))
    rows = torch.from_numpy(g.standard_normal((N, Hq + 2 * H, D)) * ch).to(dt)
    slots = g.permutation(pages * page)[:N].astype(np.int32)
    pos = g.integers(0, far - offset, N).astype(np.int32)
    gone = g.random(N) < 0.15
    slots[gone] = -1
    pos[gone & (g.random(N) < 0.7)] = -1
    cs = table(far, rot)
    if edit:
        edit(rows, slots, pos, cs)
    before = g.integers(0, 256, (pages, H, page // 16, 17 * D), dtype=np.uint8)
    wide = torch.full((N, Hq + 2 * H + (3 if strided else 0), D), 5.0, dtype=dt, device="cuda")
    wide[:, : Hq + 2 * H] = rows.cuda()
    q, k, v = wide[:, :Hq], wide[:, Hq: Hq + H], wide[:, Hq + H: Hq + 2 * H]
    if not strided:
        k, v = k.contiguous(), v.contiguous()
    c = m.KvCacheMxfp4(pages, page, H, D, data=torch.from_numpy(before).cuda())
    args = (c, q if Hq else None, k, v, i32(pos), i32(slots), torch.from_numpy(cs).cuda())
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    got = m.kv_append_rope_mxfp4(*args, interleaved=pairs, position_offset=offset, stream=stream)
    torch.cuda.synchronize()
    want, want_q = before.copy(), np.zeros((N, Hq, D), np.float32)
    for i in range(N):
        if pos[i] < 0:
            continue
        p = int(pos[i]) + offset
        turn = lambda x: block.rotate(x.float().numpy(), cs[p], pairs) if p < far else np.full(x.shape, np.nan, np.float32)  # noqa: E731
        want_q[i] = turn(rows[i, :Hq])
        if not 0 <= slots[i] < pages * page:
            continue
        kc, ks = ref.quantize(turn(rows[i, Hq: Hq + H]))
        vc, vs = ref.quantize(rows[i, Hq + H:].float().numpy())
        for h in range(H):
            ref.write(want, slots[i], h, kc[h], ks[h], vc[h], vs[h])
    if Hq:
        w = torch.from_numpy(want_q).bfloat16()
        nan = torch.isnan(w)
        assert torch.equal(torch.isnan(got.cpu()), nan)
        assert torch.equal(got.cpu()[~nan].view(torch.int16), w[~nan].view(torch.int16))
    else:
        assert got is None
    assert np.array_equal(c.data.cpu().numpy(), want)


@pytest.mark.parametrize("D,rot", [(64, 16), (64, 32), (64, 48), (64, 64), (128, 16), (128, 64), (128, 112), (128, 128)])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("f32", [False, True])
def test_rotations(m, D, rot, pairs, f32):
    case(m, 37, 6, 3, D, rot, f32=f32, pairs=pairs)


@pytest.mark.parametrize("N", [1, 2, 3, 15, 64, 333])
@pytest.mark.parametrize("Hq,H", [(0, 1), (1, 1), (3, 1), (4, 2), (5, 5), (28, 4), (64, 1), (7, 7)])
def test_sizes(m, N, Hq, H):
    case(m, N, Hq, H, 128 if Hq % 2 else 64, 32, page=64, seed=1)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("pairs", [False, True])
def test_slices_of_a_projection_and_offset(m, f32, pairs):
    case(m, 50, 8, 2, 128, 128, f32=f32, pairs=pairs, strided=True, offset=300, seed=2)


def test_positions_past_the_table_and_bad_slots(m):
    def edit(rows, slots, pos, cs):
        pos[:6] = [699, 700, 2 ** 31 - 1, -2 ** 31, -1, 0]
        slots[:6] = [0, 1, 2, 3, 4, 5]
        slots[6:8] = [2 ** 31 - 1, -2 ** 31]
        rest = slots[8:]
        rest[(rest >= 0) & (rest < 6)] = -1

    case(m, 20, 4, 2, 64, 64, edit=edit, seed=3)
    case(m, 20, 4, 2, 64, 64, edit=edit, seed=3, offset=1)


def test_huge_small_and_not_finite_rows(m):
    def edit(rows, slots, pos, cs):
        for i, f in enumerate((2.0 ** 120, 2.0 ** -120, 0.0, float("nan"), float("inf"), 2.0 ** -133)):
            if f in (float("nan"), float("inf")):
                rows[i, :, 5] = f
            else:
                rows[i] = rows[i] * f

    for f32 in (False, True):
        case(m, 24, 3, 2, 128, 128, f32=f32, edit=edit, seed=4)


def test_many_tokens_share_the_grid(m):
    case(m, 3001, 9, 2, 64, 64, page=128, seed=5)


def test_rows_beside_ties(m):
    """Keys whose rotated values fall on the quantiser's borders: angle 0 and values halfway between codes."""
    def edit(rows, slots, pos, cs):
        pos[pos >= 0] = 0
        grid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
        rows[:, :, :] = grid.repeat(rows.shape[2] // 8) * (1 - 2 * (torch.arange(rows.shape[2]) % 3 == 0).float())

    case(m, 16, 2, 2, 64, 64, edit=edit, seed=6)


def test_other_stream(m):
    case(m, 40, 4, 2, 128, 128, stream=torch.cuda.Stream(), seed=7)


def test_captured(m):
    c = m.KvCacheMxfp4(4, 16, 2, 64, data=torch.zeros(4, 2, 1, 17 * 64, dtype=torch.uint8, device="cuda"))
    x = torch.randn(5, 8, 64, device="cuda").bfloat16()
    pos, slots, cs = i32([0, 1, 2, 3, 4]), i32([3, 20, 33, -1, 50]), torch.from_numpy(table(100, 64)).cuda()
    q = torch.empty(5, 4, 64, dtype=torch.bfloat16, device="cuda")
    args = (c, x[:, :4], x[:, 4:6], x[:, 6:], pos, slots, cs)
    m.kv_append_rope_mxfp4(*args, q_out=q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.kv_append_rope_mxfp4(*args, q_out=q)
    x.copy_(torch.randn(5, 8, 64, device="cuda").bfloat16())
    pos.add_(40)
    slots.copy_(i32([9, 21, -1, 34, 51]))
    graph.replay()
    got, data = q.clone(), c.data.clone()
    m.kv_append_rope_mxfp4(*args, q_out=q)
    assert torch.equal(got, q) and torch.equal(data, c.data)
    want = block.rotate(x[1, :4].float().cpu().numpy(), table(100, 64)[41])
    assert torch.equal(q[1].cpu(), torch.from_numpy(want).bfloat16())


def test_refusals(m):
    c = m.KvCacheMxfp4(4, 16, 2, 64)
    x = torch.zeros(5, 8, 64, device="cuda", dtype=torch.bfloat16)
    pos, slots, cs = i32([0] * 5), i32([-1] * 5), torch.zeros(10, 64, device="cuda")

    def call(q=x[:, :4], k=x[:, 4:6], v=x[:, 6:], pos=pos, slots=slots, cs=cs, **kw):
        return m.kv_append_rope_mxfp4(c, q, k, v, pos, slots, cs, **kw)

    for kw, e in ((dict(cs=cs[:, :24].contiguous()), m.MoeError), (dict(cs=torch.zeros(10, 80, device="cuda")), m.MoeError),
                  (dict(cs=cs[:0]), m.MoeError), (dict(cs=cs.double()), TypeError), (dict(cs=cs[:, :32]), ValueError),
                  (dict(position_offset=-1), m.MoeError), (dict(q=x[:4, :4]), ValueError), (dict(q=x[:, :4].float()), TypeError),
                  (dict(pos=pos.long()), TypeError), (dict(slots=slots[:4]), ValueError), (dict(k=x[:, :3]), ValueError),
                  (dict(q=x[:, :8:2]), ValueError), (dict(q=None, q_out=x), ValueError),
                  (dict(q=x[:, :4].contiguous(), q_out=None, pos=pos, v=x[:, 6:].float()), TypeError)):
        with pytest.raises(e):
            call(**kw)
    q = x[:, :4].contiguous()
    with pytest.raises(m.MoeError, match="OVERLAP"):
        call(q=q, q_out=q)
    assert call(q=x[:0, :4], k=x[:0, 4:6], v=x[:0, 6:], pos=pos[:0], slots=slots[:0]).shape == (0, 4, 64)
    torch.cuda.synchronize()
