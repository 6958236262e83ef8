"""The rest of the attention block on 4-bit weights and cache, as measured workloads.

Three operators of a decoder layer, next to the MoE layer and the 4-bit KV
cache: a dense linear layer on MXFP4 weights with bias, activation and residual
in its epilogue (``linear_a16w4_mxfp4``), the position rotation of queries and
keys on the way into the quantising cache write (``kv_append_rope_mxfp4``), and
attention of a batch whose requests share a cached prefix, which is read once
for all of them (``attention_kv_mxfp4_shared``).  Each case is run in a plain form
(elementary torch operations, float32) or, with ``own`` set, through the package.

MXFP4: 32 consecutive values along a row share a scale byte s (value code *
2^(s - 127)), two E2M1 codes a byte, the even element in the low nibble.  A
weight is uint8 [N, K / 2] with scales uint8 [N, K / 32].  The cache is uint8
[pages, kv heads, page_size / 16, 17 * D], one record per 16 tokens and head;
with NB = D / 32 scale blocks per row, a record holds
  K codes  [half 2][g 8][t 4][NB][4]        token 8*half + g, row byte 16*b + 4*t + j
  V codes  [hi 2][g 8][t 4][lo 2][NB][2]    token 8*hi + 2*t + lo, row byte 16*b + 2*g + j
  K scales [16][NB], V scales [16][NB]
"""

import itertools
import math
import random

import torch

own = False

LUT = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ------------------------------------------------------------------ cases


def listed():
    return [
        # the fused q/k/v projection of one decoding token (28 + 2 * 4 heads of 128, hidden 3584): latency
        dict(name="linear 1 qkv", op="linear", T=1, K=3584, N=4608, act="none", bias=True, res=False, f32=False, strided=False),
        # the output projection of a small decoding batch, added to the residual stream
        dict(name="linear 32 out", op="linear", T=32, K=3584, N=3584, act="none", bias=False, res=True, f32=False, strided=True),
        # a scheduler step of mixed requests through a plain MLP's up projection
        dict(name="linear 250 up", op="linear", T=250, K=3584, N=8192, act="silu", bias=True, res=False, f32=False, strided=False),
        # odd sizes: a classifier head's logits in float32 from slices of wider rows
        dict(name="linear 1003 odd", op="linear", T=1003, K=2080, N=1111, act="gelu", bias=True, res=True, f32=True, strided=True),
        # a prompt batch through the gated half of a shared expert
        dict(name="linear 8192 gated", op="linear", T=8192, K=3584, N=7168, act="swiglu", bias=False, res=False, f32=False, strided=False),
        # one new token of each of 32 decoding requests, rotated and written
        dict(name="rope 32 decode", op="rope", N=32, Hq=28, Hkv=4, D=128, rot=128, page=64, f32=False, pairs=False, skip=0.0, far=131072),
        # a prompt chunk: queries, keys and values are slices of one projection's rows
        dict(name="rope 16384 prompt", op="rope", N=16384, Hq=28, Hkv=4, D=128, rot=128, page=64, f32=False, pairs=False, skip=0.0, far=32768),
        # float32 rows, a quarter of each head rotated in neighbouring pairs, heads of 64, padding tokens among them
        dict(name="rope 5003 pairs f32", op="rope", N=5003, Hq=15, Hkv=5, D=64, rot=16, page=16, f32=True, pairs=True, skip=0.1, far=8192),
        # a few users behind one long document: few rows, the work split along the prefix
        dict(name="shared 4 x 100000", op="shared", R=4, Hq=28, Hkv=4, D=128, page=64, P=100003, ctx=500, q=1, even=False, dead=0.0, lse=False),
        # a serving batch behind a long system prompt
        dict(name="shared 64 x 32768", op="shared", R=64, Hq=28, Hkv=4, D=128, page=64, P=32768, ctx=2048, q=1, even=False, dead=0.0, lse=True),
        # a large batch behind a shorter one
        dict(name="shared 256 x 8192", op="shared", R=256, Hq=28, Hkv=4, D=128, page=64, P=8192, ctx=1024, q=1, even=False, dead=0.0, lse=False),
        # draft tokens verified per request, heads of 64, a prefix that ends inside a page, empty places in the batch
        dict(name="shared 24 x 4 verify", op="shared", R=24, Hq=32, Hkv=8, D=64, page=16, P=5003, ctx=700, q=4, even=False, dead=0.2, lse=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    kind = rng.choice(("linear", "linear", "rope", "shared", "shared"))
    D, page = rng.choice((64, 128, 128)), rng.choice((16, 32, 64, 128))
    if kind == "linear":
        act = rng.choice(("none", "none", "silu", "gelu", "swiglu"))
        c = dict(op="linear", T=_log(rng, 1, 8192), K=32 * _log(rng, 1, 256), N=_log(rng, 16, 8192), act=act,
                 bias=rng.random() < 0.5, res=rng.random() < 0.5, f32=rng.random() < 0.2, strided=rng.random() < 0.4)
        # no more products than the largest listed case
        c["T"] = max(1, min(c["T"], 8192 * 3584 * 7168 // (c["K"] * c["N"])))
        if act == "swiglu":
            c["N"] += c["N"] % 2
        return c
    if kind == "rope":
        Hkv = rng.randint(1, 8)
        return dict(op="rope", N=_log(rng, 1, 10000), Hq=Hkv * rng.choice((1, 2, 3, 4, 7, 8)), Hkv=Hkv, D=D,
                    rot=rng.choice((D, D, D // 2, 16, 48)), page=page, f32=rng.random() < 0.3, pairs=rng.random() < 0.4,
                    skip=rng.choice((0.0, rng.uniform(0, 0.5))), far=_log(rng, 64, 131072))
    Hkv = rng.choice((1, 2, 3, 4, 8))
    G = rng.choice((1, 2, 4, 5, 7, 8, 12, 16))
    c = dict(op="shared", R=_log(rng, 1, 256), Hq=Hkv * G, Hkv=Hkv, D=D, page=page, P=1, ctx=1,
             q=rng.choice((1, 1, 1, rng.randint(2, 8), rng.randint(9, 64))), even=rng.random() < 0.3,
             dead=rng.choice((0.0, 0.0, rng.uniform(0, 0.4))), lse=rng.random() < 0.5)
    # scores and cached values within those of the large listed batches
    room = 64 * 28 * 32768 // (c["R"] * c["q"] * c["Hq"])
    c["P"] = _log(rng, 1, max(2, min(131072, room, 131072 * 4 * 128 // (Hkv * D))))
    c["ctx"] = max(c["q"], _log(rng, 1, max(2, min(8192, 64 * 2048 * 4 * 128 // (c["R"] * Hkv * D), max(1, room - c["P"])))))
    return c


def _lens(c):
    """The case's request lengths, from its sizes alone: own tokens (the step's included) per request, -1 for an empty place."""
    r = random.Random("%d %d %d %d" % (c["R"], c["ctx"], c["q"], c["P"]))
    out = []
    for i in range(c["R"]):
        n = c["ctx"] if c["even"] or i == 0 else r.randint(c["q"], max(c["q"], c["ctx"]))
        out.append(-1 if i and r.random() < c["dead"] else n)
    return out


def work(case):
    c = case
    if c["op"] == "linear":
        T, K, N = c["T"], c["K"], c["N"]
        cols = N // 2 if c["act"] == "swiglu" else N
        size = 4 if c["f32"] else 2
        return {"bytes": N * K * 17 // 32 + 2 * T * K + size * T * cols + (2 * N if c["bias"] else 0) + (2 * T * cols if c["res"] else 0),
                "flops": 2 * T * K * N}
    if c["op"] == "rope":
        live = 1 - c["skip"]
        size = 4 if c["f32"] else 2
        rows = c["Hq"] + 2 * c["Hkv"] * live
        # rows in, rotated queries out, codes and scales out and read once, keys and values back, table rows, slots and positions
        return {"bytes": int(c["N"] * (c["D"] * (size * rows + 2 * c["Hq"] + 2 * c["Hkv"] * (2 * 17 / 32 * live + 2))
                                       + 4 * c["rot"] + 12)),
                "flops": int(3 * c["N"] * (c["Hq"] + c["Hkv"] * live) * c["rot"])}
    lens, q = _lens(c), c["q"]
    live = sum(n >= 0 for n in lens)
    keys = c["P"] + sum(max(n, 0) for n in lens)
    seen = sum(q * c["P"] + q * n - q * (q - 1) // 2 for n in lens if n >= 0)
    return {"bytes": keys * c["Hkv"] * c["D"] * 34 // 32 + 4 * live * q * c["Hq"] * c["D"] + (4 * live * q * c["Hq"] if c["lse"] else 0),
            "flops": 4 * c["D"] * c["Hq"] * seen}


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _two(s):
    """2^(s - 127) as float32 for whole s in [0, 254], exact (s = 0 is subnormal)."""
    s = s.to(torch.int32)
    return torch.where(s > 0, s << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _codes_of(x):
    """MXFP4 of float32 rows [..., D]: (bytes [..., D/2], scale bytes [..., D/32]) as uint8."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    e = torch.frexp(amax)[1] - 1
    s = torch.where(amax < 2.0 ** -125, torch.zeros_like(e), e - 2 + 127)
    r = b * _two(254 - s)[..., None]
    a = r.abs()
    # nearest of 0 .5 1 1.5 2 3 4 6, ties to the even code
    m = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = m + 8 * torch.signbit(r)
    code = code.flatten(-2).unflatten(-1, (-1, 2))
    return (code[..., 0] + 16 * code[..., 1]).to(torch.uint8), s.to(torch.uint8)


def _records_of(kc, ks, vc, vs):
    """Records [n, 17 D] of n groups of 16 tokens: codes [n, 16, D/2], scales [n, 16, D/32]."""
    n, NB = kc.shape[0], ks.shape[-1]
    k = kc.view(n, 2, 8, NB, 4, 4).permute(0, 1, 2, 4, 3, 5).reshape(n, -1)
    v = vc.view(n, 2, 4, 2, NB, 8, 2).permute(0, 1, 5, 2, 3, 4, 6).reshape(n, -1)
    return torch.cat([k, v, ks.reshape(n, -1), vs.reshape(n, -1)], 1)


def _rows_like_model(g, n, D, dtype=torch.float32):
    """Rows as a projection gives them: Gaussian, channels of unlike size, a few rows much smaller or larger."""
    ch = torch.exp(0.6 * torch.randn(D, generator=g, device="cuda"))
    tok = torch.exp(0.5 * torch.randn(n, 1, generator=g, device="cuda"))
    return (torch.randn(n, D, generator=g, device="cuda") * ch * tok).to(dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = {"case": dict(c)}
    return {"linear": _prepare_linear, "rope": _prepare_rope, "shared": _prepare_shared}[c["op"]](c, g, st)


def _prepare_linear(c, g, st):
    T, K, N = c["T"], c["K"], c["N"]
    cols = N // 2 if c["act"] == "swiglu" else N
    wide = 64 if c["strided"] else 0  # rows are slices of wider ones
    x = _rows_like_model(g, T, K + wide, torch.bfloat16)[:, wide // 2: wide // 2 + K]
    # a trained matrix: Gaussian, rows of unlike size
    w = torch.randn(N, K, generator=g, device="cuda") * K ** -0.5 * torch.exp(0.3 * torch.randn(N, 1, generator=g, device="cuda"))
    st["w"], st["ws"] = _codes_of(w)
    st["x"] = x
    st["bias"] = (0.3 * torch.randn(N, generator=g, device="cuda")).bfloat16() if c["bias"] else None
    st["res"] = _rows_like_model(g, T, cols + wide, torch.bfloat16)[:, :cols] if c["res"] else None
    if own:
        import mxfp4_weight_only_gb300 as m

        st["out"] = torch.empty(T, cols, dtype=torch.float32 if c["f32"] else torch.bfloat16, device="cuda")
        st["work"] = torch.zeros(m.linear_workspace_bytes(T, N, K), dtype=torch.uint8, device="cuda")
    return st


def _prepare_rope(c, g, st):
    N, Hq, Hkv, D, p = c["N"], c["Hq"], c["Hkv"], c["D"], c["page"]
    pages = -(-N // p) + 7
    rows = _rows_like_model(g, N, (Hq + 2 * Hkv) * D, torch.float32 if c["f32"] else torch.bfloat16)
    q, k, v = (x.unflatten(1, (-1, D)) for x in rows.split((Hq * D, Hkv * D, Hkv * D), 1))
    # cosines and sines of every position, as a model keeps them
    f = 10000.0 ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"])
    a = torch.arange(c["far"], device="cuda", dtype=torch.float64)[:, None] * f
    table = torch.cat([a.cos(), a.sin()], 1).float()
    # tokens of several requests at any position; padding tokens have slot and position -1
    pos = torch.randint(0, c["far"], (N,), generator=g, device="cuda", dtype=torch.int32)
    perm = torch.randperm(pages, generator=g, device="cuda")
    t = torch.arange(N, device="cuda") + int(torch.randint(0, p, (1,), generator=g, device="cuda"))
    slots = (perm[t // p] * p + t % p).to(torch.int32)
    gone = torch.rand(N, generator=g, device="cuda") < c["skip"]
    slots[gone] = -1
    pos[gone] = -1
    data = torch.randint(0, 255, (pages, Hkv, p // 16, 17 * D), generator=g, device="cuda", dtype=torch.uint8)
    st.update(q=q, k=k, v=v, table=table, pos=pos, slots=slots, data=data)
    if own:
        import mxfp4_weight_only_gb300 as m

        st["cache"] = m.KvCacheMxfp4(pages, p, Hkv, D, data=data)
        st["q_out"] = torch.empty(N, Hq, D, dtype=torch.bfloat16, device="cuda")
        st["out"] = tuple(torch.empty(N, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    return st


def _prepare_shared(c, g, st):
    D, Hkv, p, R, q = c["D"], c["Hkv"], c["page"], c["R"], c["q"]
    lens = _lens(c)
    blocks = [-(-max(n, 0) // p) for n in lens]
    first = -(-c["P"] // p)  # pages of the prefix
    mb, pages = max(1, max(blocks)), first + sum(blocks) + 3
    # records drawn from a pool of quantised rows
    pool = 1024
    codes = [_codes_of(_rows_like_model(g, pool * 16, D)) for _ in range(2)]
    rec = _records_of(codes[0][0].view(pool, 16, -1), codes[0][1].view(pool, 16, -1),
                      codes[1][0].view(pool, 16, -1), codes[1][1].view(pool, 16, -1))
    n_rec = pages * Hkv * (p // 16)
    data = rec[torch.randint(0, pool, (n_rec,), generator=g, device="cuda")].view(pages, Hkv, p // 16, 17 * D)
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = perm[:first].clone()
    bt = torch.full((R, mb), -1, dtype=torch.int32, device="cuda")
    held = torch.arange(mb, device="cuda")[None, :] < _ints(blocks)[:, None]
    bt[held] = perm[first: first + sum(blocks)]
    n_k = _ints(lens)
    # slots past a length hold what earlier requests left there, not-a-number scales among it
    ends = [(int(table[-1]), c["P"])] + [(b, n) for b, n in zip(torch.gather(
        bt, 1, ((n_k - 1).clamp(min=0) // p)[:, None].long())[:, 0].tolist(), lens) if n > 0]
    last = torch.tensor([b for b, _ in ends], device="cuda")
    used = torch.tensor([(n - 1) % p + 1 for _, n in ends], device="cuda")
    tail = torch.arange(p, device="cuda")[None, :] >= used[:, None]
    sc = data[last, :, :, 16 * D:].view(len(ends), Hkv, p // 16, 2, 16, D // 32)
    sc = torch.where(tail.view(len(ends), 1, p // 16, 1, 16, 1), torch.full_like(sc, 255), sc)
    data[last, :, :, 16 * D:] = sc.reshape(len(ends), Hkv, p // 16, D)
    x = (1.5 * torch.randn(R * q, c["Hq"], D, generator=g, device="cuda")).to(torch.bfloat16)
    st.update(q=x, data=data, table=table, P=_ints([c["P"]]), bt=bt, seq_lens=n_k, query_start=_ints(list(range(0, R * q + 1, q))),
              scale=D ** -0.5)
    if own:
        import mxfp4_weight_only_gb300 as m

        st["cache"] = m.KvCacheMxfp4(pages, p, Hkv, D, data=data)
        st["work"] = torch.zeros(m.attention_shared_workspace_bytes(st["cache"], R, R * q, c["Hq"], mb, q, first),
                                 dtype=torch.uint8, device="cuda")
        st["out"] = torch.empty_like(x)
        st["lse"] = torch.empty(R * q, c["Hq"], dtype=torch.float32, device="cuda") if c["lse"] else None
    return st


# ------------------------------------------------------------------ one pass


def run(state):
    st, c = state, state["case"]
    if own:
        import mxfp4_weight_only_gb300 as m

        if c["op"] == "linear":
            return m.linear_a16w4_mxfp4(st["x"], st["w"], st["ws"], bias=st["bias"], act=c["act"], residual=st["res"],
                                        out=st["out"], workspace=st["work"])
        if c["op"] == "rope":
            q = m.kv_append_rope_mxfp4(st["cache"], st["q"], st["k"], st["v"], st["pos"], st["slots"], st["table"],
                                       interleaved=c["pairs"], q_out=st["q_out"])
            k, v = m.kv_gather_mxfp4(st["cache"], st["slots"], k_out=st["out"][0], v_out=st["out"][1])
            return {"q": q, "k": k, "v": v}
        out = m.attention_kv_mxfp4_shared(st["q"], st["cache"], st["table"], st["P"], st["bt"], st["seq_lens"],
                                          st["query_start"], c["q"], scale=st["scale"], out=st["out"], lse=st["lse"],
                                          workspace=st["work"])
        return {"out": out} if st["lse"] is None else {"out": out, "lse": st["lse"]}
    return {"linear": _plain_linear, "rope": _plain_rope, "shared": _plain_shared}[c["op"]](st)


def _values_of(codes, scales):
    """float32 values of bytes [..., D/2] and scale bytes [..., D/32]."""
    lut = torch.tensor(LUT, device=codes.device)
    pair = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    two = torch.where(scales == 255, float("nan"), _two(scales))
    return (lut[pair.int()].unflatten(-1, (-1, 32)) * two[..., None]).flatten(-2)


def _plain_linear(st):
    c = st["case"]
    h = torch.matmul(st["x"].float(), _values_of(st["w"], st["ws"]).t())
    if st["bias"] is not None:
        h = h + st["bias"].float()
    if c["act"] == "swiglu":
        a, b = h.chunk(2, 1)
        h = a / (1 + torch.exp(-a)) * b
    elif c["act"] == "silu":
        h = h / (1 + torch.exp(-h))
    elif c["act"] == "gelu":
        h = 0.5 * h * (1 + torch.erf(h * 0.5 ** 0.5))
    if st["res"] is not None:
        h = h + st["res"].float()
    return h if c["f32"] else h.to(torch.bfloat16)


def _places(D, dev):
    """Byte of a record that holds byte j of token t's K row and V row: two int64 [16, D/2]."""
    NB = D // 32
    i = torch.arange(8 * D, device=dev)
    k = i.view(2, 8, 4, NB, 4).permute(0, 1, 3, 2, 4).reshape(16, D // 2)
    v = i.view(2, 8, 4, 2, NB, 2).permute(0, 2, 3, 4, 1, 5).reshape(16, D // 2)
    return k, 8 * D + v


def _slot_bytes(slots, data, D):
    """Flat cache bytes of each slot and head: K codes, V codes, K scales, V scales as int64 [N, H, ...]."""
    P, H, gp, rec = data.shape
    s = slots.long().clamp(min=0)
    page, off = s // (16 * gp), s % (16 * gp)
    base = ((page[:, None] * H + torch.arange(H, device=s.device)) * gp + (off // 16)[:, None])[..., None] * rec
    pk, pv = _places(D, s.device)
    o = off % 16
    ks = 16 * D + o[:, None] * (D // 32) + torch.arange(D // 32, device=s.device)
    return base + pk[o][:, None], base + pv[o][:, None], base + ks[:, None], base + (ks + D // 2)[:, None]


def _turn(x, cos, sin, rot, pairs):
    """Rows [N, H, D] with their first ``rot`` elements rotated in pairs, each product and sum in float32."""
    x = x.float()
    y = x[..., :rot]
    a, b = (y[..., 0::2], y[..., 1::2]) if pairs else y.chunk(2, -1)
    c, d = a * cos - b * sin, b * cos + a * sin
    z = torch.stack([c, d], -1).flatten(-2) if pairs else torch.cat([c, d], -1)
    return torch.cat([z, x[..., rot:]], -1)


def _plain_rope(st):
    c, data, slots, D = st["case"], st["data"], st["slots"], st["case"]["D"]
    cos, sin = st["table"][st["pos"].long().clamp(min=0)][:, None].chunk(2, -1)
    live = (slots >= 0)[:, None, None]
    q = torch.where(live, _turn(st["q"], cos, sin, c["rot"], c["pairs"]), 0.0).to(torch.bfloat16)
    kc, ks = _codes_of(_turn(st["k"], cos, sin, c["rot"], c["pairs"]))
    vc, vs = _codes_of(st["v"].float())
    flat = data.view(-1)
    bk, bv, bks, bvs = _slot_bytes(slots, data, D)
    # a token without a slot repeats the write of the first one that has a slot (or rewrites what is there)
    one = live.int().argmax(0)[0, 0]
    at = torch.cat([torch.where(live, i, i[one]).flatten() for i in (bk, bv, bks, bvs)])
    what = torch.cat([torch.where(live, x, torch.where(live.any(), x[one], flat[i[one]])).flatten()
                      for i, x in ((bk, kc), (bv, vc), (bks, ks), (bvs, vs))])
    flat[at] = what
    out = [torch.where(live, _values_of(flat[i], flat[j]), 0.0).to(torch.bfloat16) for i, j in ((bk, bks), (bv, bvs))]
    return {"q": q, "k": out[0], "v": out[1]}


def _dense(data, pages, D):
    """Keys and values on ``pages`` [R, blocks] (-1: none), float32 [R, H, keys, D]."""
    R, mb = pages.shape
    H, S, NB = data.shape[1], mb * data.shape[2] * 16, D // 32
    rec = data[pages.long().clamp(min=0)].permute(0, 2, 1, 3, 4).reshape(R, H, S // 16, 17 * D)
    at = _places(D, data.device)
    codes = [rec[..., i.flatten()].unflatten(-1, (16, D // 2)).reshape(R, H, S, D // 2) for i in at]
    scales = rec[..., 16 * D:].reshape(R, H, S // 16, 2, 16, NB)
    return [_values_of(codes[i], scales[:, :, :, i].reshape(R, H, S, NB)) for i in (0, 1)]


def _plain_shared(st):
    c, D, Hkv, Hq, R, Q = st["case"], st["case"]["D"], st["case"]["Hkv"], st["case"]["Hq"], st["case"]["R"], st["case"]["q"]
    G, n = Hq // Hkv, st["seq_lens"].long()
    q = st["q"].float().view(R, Q, Hkv, G, D).permute(2, 0, 3, 1, 4)  # [Hkv, R, G, Q, D]
    # the prefix: one set of keys for all rows
    k, v = _dense(st["data"], st["table"][None], D)
    there = torch.arange(k.shape[2], device=n.device) < st["P"][:, None]
    k, v = (torch.where(there[:, None, :, None], x, 0.0)[0] for x in (k, v))
    s0 = torch.matmul(q.reshape(Hkv, -1, D), k.transpose(1, 2)).mul_(st["scale"])
    s0 = s0.masked_fill_(~there[:, None], float("-inf")).unflatten(1, (R, G, Q))
    # each request's own keys
    k1, v1 = _dense(st["data"], st["bt"], D)
    key = torch.arange(k1.shape[2], device=n.device)
    there = key < n[:, None]
    k1, v1 = (torch.where(there[:, None, :, None], x, 0.0) for x in (k1, v1))
    s1 = torch.matmul(q.transpose(0, 1).flatten(2, 3), k1.transpose(2, 3)).mul_(st["scale"]).unflatten(2, (G, Q))
    pos = n[:, None] - Q + torch.arange(Q, device=n.device)
    see = there[:, None] & (key <= pos[..., None])
    s1 = s1.masked_fill_(~see[:, None, None], float("-inf")).transpose(0, 1)
    # an empty place in the batch sees nothing
    dead = (n < 0)[None, :, None, None, None]
    s0 = s0.masked_fill_(dead, float("-inf"))
    m = torch.maximum(s0.amax(-1, keepdim=True), s1.amax(-1, keepdim=True))
    m = torch.where(m == float("-inf"), 0.0, m)
    e0, e1 = s0.sub_(m).exp_(), s1.sub(m).exp_()
    l = e0.sum(-1, keepdim=True) + e1.sum(-1, keepdim=True)
    o = torch.matmul(e0.flatten(1, 3), v).unflatten(1, (R, G, Q))
    o = o + torch.matmul(e1.transpose(0, 1).flatten(2, 3), v1).unflatten(2, (G, Q)).transpose(0, 1)
    o = o / torch.where(l == 0, 1.0, l)
    lse = torch.where(l == 0, float("-inf"), m + torch.log(l))[..., 0]
    out = o.permute(1, 3, 0, 2, 4).reshape(R * Q, Hq, D).to(torch.bfloat16)
    return {"out": out, "lse": lse.permute(1, 3, 0, 2).reshape(R * Q, Hq)} if c["lse"] else {"out": out}


# ------------------------------------------------------------------ the definition in 64 bits


def _pow2(e):
    """2^e in float64 for whole e, exact."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_values(codes, scales):
    """float64 values of code numbers [..., D] and scale bytes [..., D/32]."""
    mant, ex = codes % 2, codes // 2 % 4
    val = torch.where(ex == 0, mant * 0.5, (1 + mant * 0.5) * _pow2(ex - 1))
    return torch.where(codes >= 8, -val, val).double() * _pow2(scales.long() - 127).repeat_interleave(32, -1)


def _exact_rows(data, page, head, n, which, D):
    """float64 rows [n, D] of the first n tokens on the pages ``page`` of one head; which: 0 keys, 1 values."""
    NB = D // 32
    recs = data[page.long(), head].reshape(-1, 17 * D)[: -(-n // 16)]
    tok = torch.arange(16, device=data.device)[:, None]
    byte = torch.arange(D // 2, device=data.device)[None, :]
    b, w = byte // 16, byte % 16
    if which == 0:
        at = ((tok * 4 + w // 4) * NB + b) * 4 + w % 4
    else:
        at = 8 * D + (((((tok // 8) * 8 + w // 2) * 4 + tok % 8 // 2) * 2 + tok % 2) * NB + b) * 2 + w % 2
    by = recs[:, at.reshape(-1)].reshape(-1, D // 2)[:n].long()
    sc = recs[:, 16 * D + which * (D // 2): 16 * D + (which + 1) * (D // 2)].reshape(-1, NB)[:n]
    return _exact_values(torch.stack([by % 16, by // 16], 2).reshape(n, D), sc)


def _exact_quant(x):
    b = x.double().reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.clamp(amax, min=2.0 ** -125)))
    # the logarithm may be off by its last bit at a power of two
    e = torch.where(_pow2(e) > amax, e - 1, torch.where(_pow2(e + 1) <= amax, e + 1, e))
    two = torch.where(amax < 2.0 ** -125, 2.0 ** -127, _pow2(e - 2))
    y = (b / two).abs()
    # spacing of the grid: 0.5 below 2, 1 below 4, 2 above; ties to the even multiple are ties to the even code
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    y = torch.clamp(torch.round(y / step) * step, max=6.0)
    return (torch.sign(b) * y * two).reshape(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    return {"linear": _exact_linear, "rope": _exact_rope, "shared": _exact_shared}[case["op"]](case, st)


def _exact_linear(c, st):
    T, N = c["T"], c["N"]
    outs = []
    for t in range(0, T, 1024):
        x = st["x"][t: t + 1024].double()
        h = torch.empty(len(x), N, dtype=torch.float64, device="cuda")
        for i in range(0, N, 2048):
            by = st["w"][i: i + 2048].long()
            h[:, i: i + 2048] = x @ _exact_values(torch.stack([by % 16, by // 16], 2).flatten(1), st["ws"][i: i + 2048]).t()
        if st["bias"] is not None:
            h += st["bias"].double()
        if c["act"] == "swiglu":
            h = h[:, : N // 2] * torch.sigmoid(h[:, : N // 2]) * h[:, N // 2:]
        elif c["act"] == "silu":
            h = h * torch.sigmoid(h)
        elif c["act"] == "gelu":
            h = h * 0.5 * torch.erfc(-h / math.sqrt(2))
        if st["res"] is not None:
            h = h + st["res"][t: t + 1024].double()
        outs.append(h)
    return torch.cat(outs)


def _exact_rope(c, st):
    rot, live = c["rot"], (st["slots"] >= 0)[:, None, None]
    i = torch.arange(rot // 2, device="cuda")
    first, second = (2 * i, 2 * i + 1) if c["pairs"] else (i, i + rot // 2)
    row = st["table"].double()[st["pos"].clamp(min=0).long()]
    z = torch.complex(row[:, : rot // 2], row[:, rot // 2:])[:, None]

    def turned(x):
        y = x.double().clone()
        w = torch.complex(y[..., first], y[..., second]) * z
        y[..., first], y[..., second] = w.real, w.imag
        return y

    return {"q": torch.where(live, turned(st["q"]), 0.0), "k": torch.where(live, _exact_quant(turned(st["k"])), 0.0),
            "v": torch.where(live, _exact_quant(st["v"]), 0.0)}


def _exact_shared(c, st):
    D, Hkv, Hq, p, Q, P = c["D"], c["Hkv"], c["Hq"], c["page"], c["q"], c["P"]
    G, lens = Hq // Hkv, _lens(c)
    out = torch.zeros(len(lens) * Q, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((len(lens) * Q, Hq), float("-inf"), dtype=torch.float64, device="cuda")
    for h in range(Hkv):
        k0, v0 = (_exact_rows(st["data"], st["table"], h, P, w, D) for w in (0, 1))
        for r, n in enumerate(lens):
            if n < 0:
                continue
            page = st["bt"][r, : -(-n // p)]
            k, v = (torch.cat([x, _exact_rows(st["data"], page, h, n, w, D)]) for w, x in ((0, k0), (1, v0)))
            q = st["q"][r * Q: r * Q + Q, h * G: (h + 1) * G].double().reshape(Q * G, D)
            s = (q @ k.t() * st["scale"]).view(Q, G, P + n)
            # row i may look back to the prefix and to its own position n - Q + i
            last = P + n - Q + torch.arange(Q, device="cuda")
            s = torch.where(torch.arange(P + n, device="cuda") <= last.clamp(min=P - 1)[:, None, None], s, float("-inf"))
            z = torch.logsumexp(s, -1)
            out[r * Q: r * Q + Q, h * G: (h + 1) * G] = (torch.exp(s - z[..., None]).view(Q * G, P + n) @ v).view(Q, G, D)
            lse[r * Q: r * Q + Q, h * G: (h + 1) * G] = z
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}
