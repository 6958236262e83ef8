"""The 4-bit KV cache operators as measured workloads.

Four operators of the decoder layer's attention half, next to the MoE layer:
page tables and slot maps from request lengths (``kv_page_tables``), the MXFP4
quantising cache write and its read-back (``kv_append_mxfp4``,
``kv_gather_mxfp4``), and attention over the 4-bit cache
(``attention_kv_mxfp4``).  Each case is run in a plain form (elementary torch
operations, float32) or, with ``own`` set, through the package.

Cache layout: uint8 [pages, kv heads, page_size / 16, 17 * D], one record per
16 tokens and head.  With NB = D / 32 scale blocks per row, a record holds
  K codes  [half 2][g 8][t 4][NB][4]        token 8*half + g, row byte 16*b + 4*t + j
  V codes  [hi 2][g 8][t 4][lo 2][NB][2]    token 8*hi + 2*t + lo, row byte 16*b + 2*g + j
  K scales [16][NB], V scales [16][NB]      E8M0, value 2^(s - 127)
where a row byte j holds elements 2j (low nibble) and 2j + 1 as E2M1 codes.
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
        # eight decoding requests take one token each: the table update of a small serving step
        dict(name="tables 8 decode", op="tables", R=8, page=64, ctx=4096, new_max=1, release=0.0, free=1.5),
        # a full scheduler step: 1,000 requests, a tenth of them prompts, some finished, too few free pages for all
        dict(name="tables 1000 mixed", op="tables", R=1000, page=16, ctx=8192, new_max=700, release=0.05, free=0.9),
        # one new token of each of 32 decoding requests written and read back
        dict(name="append 32 decode", op="append", N=32, Hkv=4, D=128, page=64, f32=False, skip=0.0, fused=True),
        # a prompt chunk's keys and values, slices of a fused projection, written and read back
        dict(name="append 16384 prompt", op="append", N=16384, Hkv=8, D=128, page=64, f32=False, skip=0.0, fused=True),
        # float32 rows of an odd count with padding tokens, heads of 64
        dict(name="append 5003 f32", op="append", N=5003, Hkv=5, D=64, page=16, f32=True, skip=0.1, fused=False),
        # one user, short context: latency of the smallest decode call (28 heads of 128 = hidden 3584)
        dict(name="decode 1 x 1000", op="attn", R=1, Hq=28, Hkv=4, D=128, page=64, ctx=1000, q=1, qmin=1, dec=0.0,
             even=True, window=0, causal=True, lse=False),
        # a small serving batch with ragged contexts
        dict(name="decode 32 x 8192", op="attn", R=32, Hq=28, Hkv=4, D=128, page=64, ctx=8192, q=1, qmin=1, dec=0.0,
             even=False, window=0, causal=True, lse=True),
        # a large serving batch
        dict(name="decode 256 x 8192", op="attn", R=256, Hq=28, Hkv=4, D=128, page=64, ctx=8192, q=1, qmin=1, dec=0.0,
             even=False, window=0, causal=True, lse=False),
        # two very long contexts, 16 query heads a kv head: few rows, the work split along the context
        dict(name="decode 2 x 262144", op="attn", R=2, Hq=32, Hkv=2, D=128, page=128, ctx=262139, q=1, qmin=1, dec=0.0,
             even=True, window=0, causal=True, lse=False),
        # four draft tokens verified per request, one query head a kv head, heads of 64, sliding window
        dict(name="verify 16 x 4 window", op="attn", R=16, Hq=32, Hkv=32, D=64, page=16, ctx=4096, q=4, qmin=1,
             dec=0.0, even=False, window=1024, causal=True, lse=True),
        # prompt chunks over cached prefixes in one batch with decoding requests
        dict(name="mixed 12 chunks", op="attn", R=12, Hq=28, Hkv=4, D=128, page=64, ctx=4096, q=1500, qmin=100,
             dec=0.5, even=False, window=0, causal=True, lse=False),
        # one long prompt, nothing cached before it
        dict(name="prompt 8192", op="attn", R=1, Hq=28, Hkv=4, D=128, page=64, ctx=8192, q=8192, qmin=8192, dec=0.0,
             even=True, window=0, causal=True, lse=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("tables", "append", "decode", "decode", "verify", "prompt"))
    page = rng.choice((16, 32, 64, 128))
    D = rng.choice((64, 128, 128))
    if kind == "tables":
        return dict(op="tables", R=_log(rng, 1, 1500), page=page, ctx=_log(rng, 16, 12000),
                    new_max=rng.choice((1, _log(rng, 2, 1000))), release=rng.choice((0.0, rng.uniform(0, 0.2))),
                    free=rng.uniform(0.5, 1.5))
    if kind == "append":
        Hkv = rng.randint(1, 10)
        return dict(op="append", N=_log(rng, 1, 12000), Hkv=Hkv, D=D, page=page, f32=rng.random() < 0.3,
                    skip=rng.choice((0.0, rng.uniform(0, 0.5))), fused=rng.random() < 0.5)
    Hkv = rng.choice((1, 2, 3, 4, 8))
    G = rng.choice((1, 2, 4, 5, 7, 8, 12, 16))
    c = dict(op="attn", R=1, Hq=Hkv * G, Hkv=Hkv, D=D, page=page, ctx=1, q=1, qmin=1, dec=0.0, even=rng.random() < 0.3,
             window=rng.choice((0, 0, _log(rng, 16, 4096))), causal=True, lse=rng.random() < 0.4)
    if kind in ("decode", "verify"):
        c["q"] = 1 if kind == "decode" else rng.randint(2, 8)
        c["R"] = _log(rng, 1, 256)
        # cached values of the batch within those of the large serving batch
        c["ctx"] = _log(rng, 1, max(2, min(262144, 256 * 8192 * 4 * 128 // (2 * c["R"] * Hkv * D))))
        return c
    c["R"] = _log(rng, 1, 12)
    # padded scores within a third of the long prompt's
    room = 8192 * 8192 * 28 // 3 // (c["R"] * c["Hq"])
    c["q"] = _log(rng, 9, max(10, min(4000, int(math.sqrt(room)))))
    c["qmin"] = rng.choice((1, c["q"], max(1, c["q"] // 8)))
    c["ctx"] = max(c["q"], _log(rng, c["q"], max(c["q"] + 1, min(16384, room // c["q"]))))
    c["dec"] = rng.choice((0.0, 0.0, 0.4))
    c["causal"] = rng.random() < 0.85
    if not c["causal"]:
        c["window"] = 0
    return c


def _lens(c):
    """The case's request lengths, from its sizes alone: (context with the new tokens, new tokens) per request."""
    r = random.Random("%d %d %d %d" % (c["R"], c["ctx"], c.get("q", c.get("new_max", 0)), c["page"]))
    out = []
    for i in range(c["R"]):
        if c["op"] == "tables":
            have = r.randint(0, c["ctx"])
            if r.random() < c["release"]:
                out.append((have, -1))
            else:
                new = 1 if c["new_max"] == 1 or r.random() < 0.9 else r.randint(0, c["new_max"])
                out.append((have, new))
        else:
            q = c["q"] if c["even"] or i == 0 else 1 if r.random() < c["dec"] else r.randint(min(c["qmin"], c["q"]), c["q"])
            n = c["ctx"] if c["even"] or i == 0 else max(q, int(round(math.exp(r.uniform(math.log(max(1, c["ctx"] / 64)), math.log(c["ctx"]))))))
            out.append((n, q))
    return out


def _max_blocks(c):
    most = max(n + max(q, 0) if c["op"] == "tables" else n for n, q in _lens(c))
    return -(-max(1, most) // c["page"])


def _max_tokens(c):
    n = sum(max(0, q) for _, q in _lens(c))
    return -(-max(1, n) // 64) * 64


def _visible(c, n, q):
    """Keys seen by the q rows of one request of n keys, added up."""
    if not c["causal"]:
        return n * q
    w = c["window"] or n
    q = min(q, n)  # rows before the first key see nothing
    first = n - q  # position of the first row that sees a key
    lo = min(q, max(0, w - first))  # rows that see every key before them
    return lo * (2 * first + lo + 1) // 2 + (q - lo) * w


def _read(c, n, q):
    """Keys of one request that any of its rows sees."""
    if c["causal"] and c["window"]:
        return min(n, c["window"] + q - 1)
    return n


def work(case):
    c = case
    if c["op"] == "tables":
        lens = _lens(c)
        new_blocks = sum(-(-(n + max(q, 0)) // c["page"]) - -(-n // c["page"]) for n, q in lens)
        # lengths in and out, row starts, slot and position of each token, pages taken and written
        return {"bytes": 4 * (4 * c["R"] + 2 * _max_tokens(c) + 2 * new_blocks), "flops": 0}
    if c["op"] == "append":
        vals = 2 * c["N"] * c["Hkv"] * c["D"]
        live = 1 - c["skip"]
        # rows in; codes and scales written and read once; bf16 rows out
        return {"bytes": int(vals * ((4 if c["f32"] else 2) * live + 2 * 17 / 32 * live + 2)) + 4 * c["N"], "flops": 0}
    lens = _lens(c)
    rows = sum(q for _, q in lens)
    keys = sum(_read(c, n, q) for n, q in lens)
    seen = sum(_visible(c, n, q) for n, q in lens)
    return {"bytes": keys * c["Hkv"] * c["D"] * 34 // 32 + 4 * rows * c["Hq"] * c["D"] + (4 * rows * c["Hq"] if c["lse"] else 0),
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
    if c["op"] == "tables":
        lens, p, mb = _lens(c), c["page"], _max_blocks(c)
        have = [-(-n // p) for n, _ in lens]
        need = [-(-(n + max(q, 0)) // p) - h for (n, q), h in zip(lens, have)]
        free = max(1, int(round(c["free"] * sum(need))))
        pages = sum(have) + free
        perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        # rows of the table: held pages first, stale entries after them
        bt = torch.randint(0, pages, (c["R"], mb), generator=g, device="cuda", dtype=torch.int32)
        held = torch.arange(mb, device="cuda")[None, :] < _ints(have)[:, None]
        bt[held] = perm[: sum(have)]
        head = int(torch.randint(0, pages, (1,), generator=g, device="cuda"))
        ring = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
        ring[(head + torch.arange(free, device="cuda")) % pages] = perm[sum(have):]
        st.update(cached=_ints([n for n, _ in lens]), new=_ints([q for _, q in lens]), bt=bt, ring=ring,
                  state=_ints([head, free]), max_tokens=_max_tokens(c))
        if own:
            N = st["max_tokens"]
            i32 = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
            st["bufs"] = dict(seq_lens=i32(c["R"]), query_start=i32(c["R"] + 1), slots=i32(N), positions=i32(N), ring_state_out=i32(2))
        return st
    D, Hkv, p = c["D"], c["Hkv"], c["page"]
    if c["op"] == "append":
        N = c["N"]
        pages = -(-N // p) + 7
        dtype = torch.float32 if c["f32"] else torch.bfloat16
        kv = torch.cat([_rows_like_model(g, N, Hkv * D, dtype) for _ in range(2)], 1)
        if c["fused"]:  # keys and values are slices of one projection's rows, queries before them
            kv = torch.cat([torch.zeros(N, 4 * Hkv * D, dtype=dtype, device="cuda"), kv], 1)
        k, v = (x.unflatten(1, (Hkv, D)) for x in kv[:, -2 * Hkv * D:].split(Hkv * D, 1))
        # tokens in order on shuffled pages, as a prompt's are; padding tokens have slot -1
        perm = torch.randperm(pages, generator=g, device="cuda")
        t = torch.arange(N, device="cuda") + int(torch.randint(0, p, (1,), generator=g, device="cuda"))
        slots = (perm[t // p] * p + t % p).to(torch.int32)
        slots[torch.rand(N, generator=g, device="cuda") < c["skip"]] = -1
        data = torch.randint(0, 255, (pages, Hkv, p // 16, 17 * D), generator=g, device="cuda", dtype=torch.uint8)
        st.update(k=k, v=v, slots=slots, data=data)
        if own:
            import mxfp4_weight_only_gb300 as m

            st["cache"] = m.KvCacheMxfp4(pages, p, Hkv, D, data=data)
            st["out"] = tuple(torch.empty(N, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        return st
    lens, mb = _lens(c), _max_blocks(c)
    blocks = [-(-n // p) for n, _ in lens]
    pages = sum(blocks) + 3
    # records drawn from a pool of quantised rows
    pool = 1024
    codes = [_codes_of(_rows_like_model(g, pool * 16, D)) for _ in range(2)]
    rec = _records_of(codes[0][0].view(pool, 16, -1), codes[0][1].view(pool, 16, -1),
                      codes[1][0].view(pool, 16, -1), codes[1][1].view(pool, 16, -1))
    n_rec = pages * Hkv * (p // 16)
    data = rec[torch.randint(0, pool, (n_rec,), generator=g, device="cuda")].view(pages, Hkv, p // 16, 17 * D)
    # slots past a request's length hold what earlier requests left there, not-a-number scales among it
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    bt = torch.full((c["R"], mb), -1, dtype=torch.int32, device="cuda")
    held = torch.arange(mb, device="cuda")[None, :] < _ints(blocks)[:, None]
    bt[held] = perm[: sum(blocks)]
    n_k = _ints([n for n, _ in lens])
    last = torch.gather(bt, 1, ((n_k - 1) // p)[:, None].long())[:, 0].long()
    tail = torch.arange(p, device="cuda")[None, :] >= ((n_k - 1) % p + 1)[:, None]
    NB = D // 32
    sc = data[last, :, :, 16 * D:].view(c["R"], Hkv, p // 16, 2, 16, NB)  # indexing copies: written back below
    sc = torch.where(tail.view(c["R"], 1, p // 16, 1, 16, 1), torch.full_like(sc, 255), sc)
    data[last, :, :, 16 * D:] = sc.reshape(c["R"], Hkv, p // 16, D)
    N = sum(q for _, q in lens)
    starts = [0, *itertools.accumulate(q for _, q in lens)]
    q = (1.5 * torch.randn(N, c["Hq"], D, generator=g, device="cuda")).to(torch.bfloat16)
    st.update(q=q, data=data, bt=bt, seq_lens=n_k, query_start=_ints(starts), max_q=max(x for _, x in lens), N=N,
              scale=D ** -0.5)
    if own:
        import mxfp4_weight_only_gb300 as m

        st["cache"] = m.KvCacheMxfp4(pages, p, Hkv, D, data=data)
        st["ws"] = torch.zeros(m.attention_workspace_bytes(st["cache"], c["R"], N, c["Hq"], mb, st["max_q"]),
                               dtype=torch.uint8, device="cuda")
        st["out"] = torch.empty_like(q)
        st["lse"] = torch.empty(N, c["Hq"], dtype=torch.float32, device="cuda") if c["lse"] else None
    return st


# ------------------------------------------------------------------ one pass


def run(state):
    st, op = state, state["case"]["op"]
    if own:
        import mxfp4_weight_only_gb300 as m

        if op == "tables":
            t = m.kv_page_tables(st["cached"], st["new"], st["bt"], st["ring"], st["state"], st["case"]["page"],
                                 st["max_tokens"], **st["bufs"])
            return {"block_table": st["bt"], "ring": st["ring"], "seq_lens": t.seq_lens, "query_start": t.query_start,
                    "slots": t.slots, "positions": t.positions, "ring_state": t.ring_state}
        if op == "append":
            m.kv_append_mxfp4(st["cache"], st["k"], st["v"], st["slots"])
            k, v = m.kv_gather_mxfp4(st["cache"], st["slots"], k_out=st["out"][0], v_out=st["out"][1])
            return {"k": k, "v": v}
        out = m.attention_kv_mxfp4(st["q"], st["cache"], st["bt"], st["seq_lens"], st["query_start"], st["max_q"],
                                   scale=st["scale"], causal=st["case"]["causal"], window=st["case"]["window"],
                                   out=st["out"], lse=st["lse"], workspace=st["ws"])
        return {"out": out} if st["lse"] is None else {"out": out, "lse": st["lse"]}
    return {"tables": _plain_tables, "append": _plain_append, "attn": _plain_attn}[op](st)


def _excl(x):
    return torch.cumsum(x, 0) - x


def _plain_tables(st):
    c, bt, ring = st["case"], st["bt"], st["ring"]
    p, M = c["page"], st["max_tokens"]
    R, mb = bt.shape
    C = ring.shape[0]
    cached, new = st["cached"].long(), st["new"].long()
    head, free = st["state"][0].long(), st["state"][1].long()
    n = new.clamp(min=0)
    start = _excl(n)
    have, every = (cached + p - 1) // p, (cached + n + p - 1) // p
    ok = (start + n <= M) & (every <= mb)
    need = torch.where(ok & (new >= 0), every - have, 0)
    ofs = _excl(need)
    ok = ok & ((need == 0) | (ofs + need <= free))
    need = torch.where(ok, need, 0)
    # new pages into the rows
    col = torch.arange(mb, device=bt.device)[None, :]
    fresh = (col >= have[:, None]) & (col < (have + need)[:, None])
    took = ring[(head + ofs[:, None] + col - have[:, None]) % C]
    bt.copy_(torch.where(fresh, took, bt))
    # pages of finished requests to the ring's end
    gone = torch.where(new < 0, have, 0)
    gofs = _excl(gone)
    # (an entry that is not given back lands in a spare place past the ring)
    at = torch.where(col < gone[:, None], (head + free + gofs[:, None] + col) % C, C)
    ext = torch.cat([ring, ring[:1]])
    ext[at.flatten()] = bt.flatten()
    ring.copy_(ext[:C])
    taken, back = need.sum(), gone.sum()
    total = n.sum()
    t = torch.arange(M, device=bt.device)
    r = (torch.searchsorted(start, t, right=True) - 1).clamp(min=0)
    pos = cached[r] + t - start[r]
    page = bt[r, (pos // p).clamp(max=mb - 1)].long()
    live = t < total
    slots = torch.where(live & ok[r], page * p + pos % p, -1)
    return {"block_table": bt, "ring": ring,
            "seq_lens": torch.where(new < 0, 0, torch.where(ok, cached + n, -1)).int(),
            "query_start": torch.cat([start, total[None]]).int(), "slots": slots.int(),
            "positions": torch.where(live, pos, -1).int(),
            "ring_state": torch.stack([(head + taken) % C, free - taken + back]).int()}


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


def _values_of(codes, scales):
    """float32 values of bytes [..., D/2] and scale bytes [..., D/32]."""
    lut = torch.tensor(LUT, device=codes.device)
    pair = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    two = torch.where(scales == 255, float("nan"), _two(scales))
    return (lut[pair.int()].unflatten(-1, (-1, 32)) * two[..., None]).flatten(-2)


def _plain_append(st):
    data, slots, D = st["data"], st["slots"], st["case"]["D"]
    flat = data.view(-1)
    bk, bv, bks, bvs = _slot_bytes(slots, data, D)
    live = (slots >= 0)[:, None, None]
    kc, ks = _codes_of(st["k"].float())
    vc, vs = _codes_of(st["v"].float())
    # a token without a slot repeats the write of the first one that has a slot (or rewrites what is there)
    one = live.int().argmax(0)[0, 0]
    at = torch.cat([torch.where(live, i, i[one]).flatten() for i in (bk, bv, bks, bvs)])
    what = torch.cat([torch.where(live, x, torch.where(live.any(), x[one], flat[i[one]])).flatten()
                      for i, x in ((bk, kc), (bv, vc), (bks, ks), (bvs, vs))])
    flat[at] = what
    out = [torch.where(live, _values_of(flat[i], flat[j]), 0.0).to(torch.bfloat16) for i, j in ((bk, bks), (bv, bvs))]
    return {"k": out[0], "v": out[1]}


def _plain_attn(st):
    c, data, bt = st["case"], st["data"], st["bt"]
    D, p, Hkv, Hq = c["D"], c["page"], c["Hkv"], c["Hq"]
    R, mb = bt.shape
    NB, G, Q = D // 32, Hq // Hkv, st["max_q"]
    S = mb * p
    # cache pages of every request, dense and in float32
    rec = data[bt.long().clamp(min=0)].permute(0, 2, 1, 3, 4).reshape(R, Hkv, S // 16, 17 * D)
    dense = []
    for_k, for_v = _places(D, data.device)
    codes = rec[..., for_k.flatten()].unflatten(-1, (16, D // 2)).reshape(R, Hkv, S, D // 2)
    scales = rec[..., 16 * D: 16 * D + D // 2].reshape(R, Hkv, S, NB)
    dense.append(_values_of(codes, scales))
    codes = rec[..., for_v.flatten()].unflatten(-1, (16, D // 2)).reshape(R, Hkv, S, D // 2)
    scales = rec[..., 16 * D + D // 2:].reshape(R, Hkv, S, NB)
    dense.append(_values_of(codes, scales))
    n, qs = st["seq_lens"].long(), st["query_start"].long()
    qn = qs[1:] - qs[:-1]
    key = torch.arange(S, device=n.device)
    there = (key[None, :] < n[:, None])[:, None, :, None]
    k, v = (torch.where(there, x, 0.0) for x in dense)
    row = torch.arange(Q, device=n.device)
    tok = (qs[:-1, None] + row).clamp(max=st["N"] - 1)
    q = st["q"][tok].float().unflatten(2, (Hkv, G)).permute(0, 2, 3, 1, 4).reshape(R, Hkv, G * Q, D)
    s = torch.matmul(q, k.transpose(2, 3)).mul_(st["scale"]).unflatten(2, (G, Q))
    pos = n[:, None] - qn[:, None] + row
    see = (key[None, None, :] < n[:, None, None]).expand(R, Q, S)
    if c["causal"]:
        see = see & (key <= pos[..., None])
    if c["window"]:
        see = see & (key > pos[..., None] - c["window"])
    s = s.masked_fill_(~see[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    m0 = torch.where(m == float("-inf"), 0.0, m)
    e = s.sub_(m0).exp_()
    l = e.sum(-1, keepdim=True)
    o = torch.matmul(e.flatten(2, 3), v).unflatten(2, (G, Q)) / torch.where(l == 0, 1.0, l)
    lse = torch.where(l == 0, float("-inf"), m0 + torch.log(l))[..., 0]
    # back to the tokens' own order
    t = torch.arange(st["N"], device=n.device)
    r = torch.searchsorted(qs[1:].contiguous(), t, right=True)
    i = t - qs[r]
    out = o.permute(0, 3, 1, 2, 4).reshape(R, Q, Hq, D)[r, i].to(torch.bfloat16)
    return {"out": out, "lse": lse.permute(0, 3, 1, 2).reshape(R, Q, Hq)[r, i]} if c["lse"] else {"out": out}


# ------------------------------------------------------------------ the definition in 64 bits


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
    sc = recs[:, 16 * D + which * (D // 2): 16 * D + (which + 1) * (D // 2)].reshape(-1, NB)[:n].double()
    code = torch.stack([by % 16, by // 16], 2).reshape(n, D)
    mag, ex = code % 2, code // 2 % 4
    val = torch.where(ex == 0, mag * 0.5, (1 + mag * 0.5) * _pow2(ex - 1))
    val = torch.where(code >= 8, -val, val).double()
    return val * _pow2(sc - 127).repeat_interleave(32, 1)


def _pow2(e):
    """2^e in float64 for whole e, exact."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


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
    c = case
    if c["op"] == "tables":
        return None  # whole numbers only
    st = prepare(case, seed)
    if c["op"] == "append":
        live = (st["slots"] >= 0)[:, None, None]
        return {x: torch.where(live, _exact_quant(st[x]), 0.0) for x in ("k", "v")}
    D, Hkv, Hq, p = c["D"], c["Hkv"], c["Hq"], c["page"]
    G = Hq // Hkv
    lens = _lens(c)
    out = torch.zeros(st["N"], Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((st["N"], Hq), float("-inf"), dtype=torch.float64, device="cuda")
    if sum(n * q for n, q in lens) * Hq * D * 4 > 1.2e13:
        return None
    at = 0
    for r, (n, qn) in enumerate(lens):
        j = torch.arange(n, device="cuda")
        page = st["bt"][r, : -(-n // p)]
        for h in range(Hkv):
            k = _exact_rows(st["data"], page, h, n, 0, D)
            v = _exact_rows(st["data"], page, h, n, 1, D)
            for i0 in range(0, qn, 1024):
                i1 = min(qn, i0 + 1024)
                pos = n - qn + torch.arange(i0, i1, device="cuda")[:, None]
                see = torch.ones(i1 - i0, n, dtype=torch.bool, device="cuda")
                if c["causal"]:
                    see = j[None, :] <= pos
                    if c["window"]:
                        see = see & (pos - j[None, :] < c["window"])
                q = st["q"][at + i0: at + i1, h * G: (h + 1) * G].double()
                s = torch.einsum("igd,jd->gij", q, k) * st["scale"]
                s = torch.where(see[None], s, float("-inf"))
                z = torch.logsumexp(s, -1)
                w = torch.where(see[None], torch.exp(s - torch.where(torch.isinf(z), 0.0, z)[..., None]), 0.0)
                out[at + i0: at + i1, h * G: (h + 1) * G] = torch.einsum("gij,jd->igd", w, v)
                lse[at + i0: at + i1, h * G: (h + 1) * G] = z.t()
        at += qn
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}
