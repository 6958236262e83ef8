"""Attention behind a shared prefix (oracle; test infrastructure only): ``kv_cache.attention``'s definition over the
prefix's keys, seen whole by every row, followed by each request's own."""

from __future__ import annotations

import numpy as np

from .kv_cache import read, values


def attention(q, data, shared, P, table, seq_lens, query_start, scale, causal=True):
    """float64 (out, lse, spread, size), as ``kv_cache.attention``."""
    q = np.asarray(q, np.float64)
    N, Hq, D = q.shape
    pages, H, gp, _ = data.shape
    p, G = 16 * gp, Hq // H
    out = np.full((N, Hq, D), np.nan)
    lse = np.full((N, Hq), np.nan)
    spread, size = np.zeros((N, Hq, D)), np.zeros((N, Hq))

    def keys(pages_of, n):
        """Values of n keys and which of them exist."""
        n = min(max(int(n), 0), len(pages_of) * p)
        j = np.arange(n)
        pg = np.asarray(pages_of)[j // p] if n else j
        there = (pg >= 0) & (pg < pages)
        kc, ks, vc, vs = read(data, np.where(there, pg, 0) * p + j % p)
        bad = (ks == 255).any(-1) | (vs == 255).any(-1)
        return n, there, bad, values(kc, np.where(ks == 255, 0, ks)), values(vc, np.where(vs == 255, 0, vs))

    first = keys(shared, P)
    for r in range(len(seq_lens)):
        q0, q1 = int(query_start[r]), int(query_start[r + 1])
        if seq_lens[r] < 0:
            out[q0:q1], lse[q0:q1] = 0.0, -np.inf
            continue
        own = keys(table[r], seq_lens[r])
        there, bad, k, v = (np.concatenate([a, b]) for a, b in zip(first[1:], own[1:]))
        j = np.arange(own[0])
        for i in range(q1 - q0):
            see = there.copy()
            if causal:
                see[first[0]:] &= j <= own[0] - (q1 - q0) + i
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
