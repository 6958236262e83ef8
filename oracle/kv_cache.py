"""The 4-bit KV cache and the attention over it (oracle; test infrastructure only).

The pages describe no cache, so these are the plain definitions:

* page tables: requests in order, a Python loop over tokens and pages;
* the write: per 32 values of a head's row the MXFP4 rule of
  ``actquant.quantize_mxfp4_act``; a block holding a NaN gets scale byte 255,
  infinities saturate to code +-6 at scale byte 252;
* records of 16 tokens of one head, 17 * D bytes, by the index formulas below;
* attention in float64: S = scale q.k, softmax over the visible keys, weighted
  sum; rows without a visible key are zero with lse -inf; a token with a scale
  byte 255 in its K or V row makes every row that sees it NaN.
"""

from __future__ import annotations

import numpy as np

from . import actquant, formats


def page_tables(cached, new, table, ring, state, page, max_tokens):
    """One step's tables.  ``table`` and ``ring`` are updated in place; returns
    (seq_lens, query_start, slots, positions, ring_state)."""
    R, mb = table.shape
    C = len(ring)
    head, free = int(state[0]), int(state[1])
    old = table.copy()
    seq = np.zeros(R, np.int32)
    start = np.zeros(R + 1, np.int32)
    slots = np.full(max_tokens, -1, np.int32)
    positions = np.full(max_tokens, -1, np.int32)
    claimed = 0  # pages asked for so far, by requests refused for want of pages too
    taken = back = 0
    for r in range(R):
        c, n = int(cached[r]), int(new[r])
        have = -(-c // page)
        start[r + 1] = start[r] + max(n, 0)
        if n < 0:
            for b in range(have):
                ring[(head + free + back) % C] = old[r, b]
                back += 1
            continue
        every = -(-(c + n) // page)
        ok = start[r] + n <= max_tokens and every <= mb and c + n <= 2 ** 31 - 1
        if ok:
            need = every - have
            ok = need == 0 or claimed + need <= free
            if ok:
                for b in range(have, every):
                    table[r, b] = ring[(head + claimed + b - have) % C]
                taken += need
            claimed += need
        seq[r] = c + n if ok else -1
        for i in range(n):
            t = start[r] + i
            if t >= max_tokens:
                break
            positions[t] = min(c + i, 2 ** 31 - 1)
            if ok:
                slots[t] = table[r, (c + i) // page] * page + (c + i) % page
    return seq, start, slots, positions, np.array([(head + taken) % C, free - taken + back], np.int32)


def quantize(x):
    """Rows [..., D] -> (codes uint8 [..., D/2], scale bytes uint8 [..., D/32]), any float values."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], -1, 32)
    nan = np.isnan(b).any(-1)
    inf = np.isinf(b).any(-1) & ~nan
    finite = np.where(np.isfinite(b), b, 0.0)
    packed, s = actquant.quantize_mxfp4_act(finite.reshape(x.shape))
    codes = formats.unpack_nibbles(packed).reshape(b.shape)
    # an infinite block: scale byte 252, the others' codes on that scale
    big, _ = _on_scale(finite, 252)
    codes = np.where(inf[..., None], np.where(np.isinf(b), 7 + 8 * (b < 0), big), codes).astype(np.uint8)
    s = np.where(nan, 255, np.where(inf, 252, s)).astype(np.uint8)
    return formats.pack_nibbles(codes.reshape(x.shape)), s


def _on_scale(v, byte):
    grid = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
    y = np.abs(v) / 2.0 ** (byte - 127)
    d = np.abs(y[..., None] - grid)
    best = d.min(-1, keepdims=True)
    code = np.where(d == best, np.arange(8) % 2 * 8 + np.arange(8), 99).argmin(-1)  # ties to the even code
    return code + 8 * np.signbit(v), y


def values(codes, scales):
    """float64 values of codes [..., D/2] and scale bytes [..., D/32]."""
    v = formats.e2m1_decode(formats.unpack_nibbles(codes))
    return v * np.repeat(formats.e8m0_decode(scales), 32, axis=-1)


def k_at(t, j, D):
    """Byte of a record that holds byte j of token t's K row."""
    return ((t * 4 + j // 4 % 4) * (D // 32) + j // 16) * 4 + j % 4


def v_at(t, j, D):
    """Byte of a record that holds byte j of token t's V row."""
    lane = (t // 8 * 8 + j % 16 // 2) * 4 + t % 8 // 2
    return 8 * D + ((lane * 2 + t % 2) * (D // 32) + j // 16) * 2 + j % 2


def write(data, slot, head, kc, ks, vc, vs):
    """Store one token's codes and scales of one head in ``data`` [pages, heads, groups, 17 D]."""
    D = data.shape[3] // 17
    NB, p = D // 32, data.shape[2] * 16
    rec = data[slot // p, head, slot % p // 16]
    t = slot % 16
    for j in range(D // 2):
        rec[k_at(t, j, D)] = kc[j]
        rec[v_at(t, j, D)] = vc[j]
    rec[16 * D + t * NB: 16 * D + (t + 1) * NB] = ks
    rec[16 * D + D // 2 + t * NB: 16 * D + D // 2 + (t + 1) * NB] = vs


def read(data, slots):
    """Codes and scales of ``slots``: K codes [n, heads, D/2], K scales, V codes, V scales."""
    D = data.shape[3] // 17
    NB, p = D // 32, data.shape[2] * 16
    slots = np.asarray(slots)
    rec = data[slots // p, :, slots % p // 16]
    t = (slots % 16)[:, None]
    j = np.arange(D // 2)[None, :]
    i, h = np.arange(len(slots))[:, None, None], np.arange(data.shape[1])[None, :, None]
    b = np.arange(NB)[None, None, :]
    ks = 16 * D + t[:, :, None] * NB + b
    return (rec[i, h, k_at(t, j, D)[:, None]], rec[i, h, ks], rec[i, h, v_at(t, j, D)[:, None]], rec[i, h, ks + D // 2])


def attention(q, data, table, seq_lens, query_start, scale, causal=True, window=0):
    """float64 (out [N, Hq, D], lse [N, Hq], spread [N, Hq, D], size [N, Hq]):
    ``spread`` is sum_j p_j |v_j| (what rounding the weights can move) and
    ``size`` the largest sum_d |scale q_d k_d| (what rounding the scores can)."""
    q = np.asarray(q, np.float64)
    N, Hq, D = q.shape
    pages, H, gp, _ = data.shape
    p, G = 16 * gp, Hq // H
    out = np.full((N, Hq, D), np.nan)
    lse = np.full((N, Hq), np.nan)
    spread, size = np.zeros((N, Hq, D)), np.zeros((N, Hq))
    for r in range(len(seq_lens)):
        n = min(max(int(seq_lens[r]), 0), table.shape[1] * p)
        q0, q1 = int(query_start[r]), int(query_start[r + 1])
        j = np.arange(n)
        pg = table[r, j // p] if n else j
        there = (pg >= 0) & (pg < pages)
        kc, ks, vc, vs = read(data, np.where(there, pg, 0) * p + j % p)
        bad = (ks == 255).any(-1) | (vs == 255).any(-1)  # [n, H]
        k = values(kc, np.where(ks == 255, 0, ks))
        v = values(vc, np.where(vs == 255, 0, vs))
        for i in range(q1 - q0):
            pos = n - (q1 - q0) + i
            see = there.copy()
            if causal:
                see &= j <= pos
                if window:
                    see &= j > pos - window
            for h in range(Hq):
                if not see.any():
                    out[q0 + i, h], lse[q0 + i, h] = 0.0, -np.inf
                    continue
                if bad[see, h // G].any():
                    continue  # NaN
                kk, vv = k[see, h // G], v[see, h // G]
                s = kk @ q[q0 + i, h] * scale
                m = s.max()
                w = np.exp(s - m)
                out[q0 + i, h] = w @ vv / w.sum()
                lse[q0 + i, h] = m + np.log(w.sum())
                spread[q0 + i, h] = w @ np.abs(vv) / w.sum()
                size[q0 + i, h] = (np.abs(kk) @ np.abs(q[q0 + i, h])).max() * abs(scale)
    return out, lse, spread, size
