"""Attention behind a shared prefix holds the weights of decoding rows as attention over the cache does: 16 bits down to 2^-126
of the largest, on the tensor cores too.

Queries and keys with one element each, so that scores are exact products.  Every 64th key of the prefix outweighs the others by
2^26 to 2^32 and has no value: results are sums of light keys alone, whose weights one f16 of p 2^9 holds as multiples of
2^-33, up to 2^-2 of them off.  The bound is that of tests/test_gpu_kv_shared.py without its term for such weights."""

import numpy as np
import pytest
import torch

from oracle import kv_cache as cache
from tests import test_gpu_kv_shared as shared
from tests.test_gpu_kv_shared import m  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def light(P, qlens, G, D, page, table, seed):
    """``table``: tokens that the shared table has room for (the choice of kernels goes by it)."""
    p = shared.problem(P, [q + 3 for q in qlens], qlens, 1, G, D, page, seed=seed, bands=((127, 127), (127, 127)), extra=0)
    g = np.random.default_rng(seed)
    rows = p["q"].shape[0]
    p["q"].zero_()
    p["q"][:, :, 5] = torch.from_numpy(g.uniform(3.7, 4.2, (rows, G))).bfloat16()
    t, byte = np.arange(16), np.arange(D // 2)
    p["data"][..., cache.k_at(t[:, None], byte, D)] = 0
    low = g.integers(1, 4, p["data"].shape[:3] + (16,)).astype(np.uint8)  # 0.5, 1, 1.5
    v = g.integers(1, 8, p["data"].shape[:3] + (16, D // 2)).astype(np.uint8)
    v |= g.integers(1, 8, v.shape).astype(np.uint8) << 4  # positive values
    heavy = np.zeros(low.shape, bool)
    for j in range(0, P, 64):
        heavy[p["shared"][j // page], :, j % page // 16, j % 16] = True
    low[heavy], v[heavy] = 7, 0
    p["data"][..., cache.k_at(t, 2, D)] = low << 4  # element 5
    p["data"][..., cache.v_at(t[:, None], byte, D)] = v
    tail = g.integers(-5, p["pages"] + 5, max(0, table // page - len(p["shared"]))).astype(np.int32)
    p["shared"] = np.concatenate([p["shared"], tail])
    p["lost"] = 2.0 ** -126 * (P + max(qlens) + 3) * 6
    return p


# slices of 257 keys and more (up to 31 of them), of at most 256, the streamed form
@pytest.mark.parametrize("P,table", [(9000, 131072), (700, 131072), (9000, 0)])
@pytest.mark.parametrize("R,q,G,D", [(40, 1, 8, 64), (33, 1, 8, 128), (20, 4, 4, 64), (1, 1, 8, 128)])
def test_light_weights(m, P, table, R, q, G, D):  # noqa: F811
    shared.both(m, light(P, [q] * R, G, D, 64, table, R), scale=1.0)


@pytest.mark.parametrize("order", ["first", "last", "between"])
@pytest.mark.parametrize("G,D", [(8, 64), (7, 128), (1, 64)])
def test_decoding_rows_beside_prompts(m, order, G, D):  # noqa: F811
    """Rows of a prompt (whose weights may have 11 bits) in the same tiles of 256 as those of decoding requests."""
    prompts, few = [-(-400 // G) + 3, -(-300 // G)], [1] * 30 + [2]
    qlens = {"first": few + prompts, "last": prompts + few, "between": prompts[:1] + few + prompts[1:]}[order]
    p = light(9000, qlens, G, D, 64, 131072, G)
    out, lse = shared.run(m, p, scale=1.0)
    mine = [r for r, q in enumerate(qlens) if q <= 2]
    rows = np.concatenate([np.arange(p["start"][r], p["start"][r + 1]) for r in mine])
    start = np.concatenate([[0], np.cumsum([qlens[r] for r in mine])])
    part = {**p, "q": p["q"][rows], "lens": p["lens"][mine], "table": p["table"][mine], "start": start}
    shared.check(part, out[rows], lse[rows], scale=1.0)
