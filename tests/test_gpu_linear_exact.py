"""Deep linear layers whose sums are exact: small whole numbers, one scale, every partial sum below 2^24, so that float32
results equal the definition whatever the order.  A value of K left out or taken twice, anywhere, shows: each
column's weights and each row's values are their own."""

import numpy as np
import pytest
import torch

from tests.test_gpu_linear import m, on_gpu  # noqa: F401
from tests.test_gpu_linear_split import splits

pytestmark = pytest.mark.gpu

GRID = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def exact(m, T, K, N, seed):  # noqa: F811
    """Values of +-1, +-2 and weights of +-1 .. +-6 (scale byte 128: twice the codes' 0.5 .. 3): sums of at most 12 K < 2^20."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.tensor([1, 2, 3, 4, 5, 9, 10, 11, 12, 13], dtype=torch.uint8)  # (none is 0)
    w = codes[torch.randint(0, 10, (N, K), generator=g)]
    x = torch.tensor([-2.0, -1, 1, 2])[torch.randint(0, 4, (T, K), generator=g)].bfloat16()
    b = torch.randint(-50, 50, (N,), generator=g).bfloat16()
    r = torch.randint(-50, 50, (T, N), generator=g).bfloat16()
    packed = w[:, 0::2] | w[:, 1::2] << 4
    out = m.linear_a16w4_mxfp4(on_gpu(x), packed.cuda(), torch.full((N, K // 32), 128, dtype=torch.uint8, device="cuda"),
                               bias=b.cuda(), residual=r.cuda(), out_dtype=torch.float32)
    want = torch.empty(T, N, dtype=torch.float64, device="cuda")
    for i in range(0, N, 512):  # (products and sums of whole numbers below 2^53)
        want[:, i: i + 512] = x.cuda().double() @ (2 * GRID.cuda()[w[i: i + 512].cuda().int()]).t()
    want += b.cuda().double() + r.cuda().double()
    bad = out.double() != want
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())
    # (the check can tell: a block less changes nearly every result)
    lost = want - x[:, -32:].cuda().double() @ (2 * GRID.cuda()[w[:, -32:].cuda().int()]).t()
    assert (lost != want).double().mean() > 0.9


DEPTHS = [96, 1056, 2080, 3232, 8224, 32768, 65536]


@pytest.mark.parametrize("K", DEPTHS)
@pytest.mark.parametrize("T,N", [(1, 5), (9, 21), (16, 33), (24, 70), (32, 5), (33, 40), (100, 65), (300, 5)])
def test_from_registers(m, T, N, K):  # noqa: F811
    assert splits(m, T, K, N) == 0
    exact(m, T, K, N, K + T)


@pytest.mark.parametrize("K", DEPTHS)
@pytest.mark.parametrize("T", [1, 9])
def test_walked(m, T, K):  # noqa: F811
    exact(m, T, K, 5000, K + T)


@pytest.mark.parametrize("n,T,K,N", [
    (2, 260, 1312, 1250), (2, 400, 2048, 800), (3, 40, 2080, 2500), (3, 300, 2592, 600), (4, 40, 3232, 2500), (4, 150, 8224, 1250),
    (4, 300, 32768, 600), (4, 256, 65536, 700), (3, 250, 65536, 5300), (2, 250, 65536, 8000), (1, 700, 1056, 4000), (1, 700, 8224, 7000),
    (1, 600, 65536, 6500), (1, 1100, 2080, 5000)])
def test_on_the_tensor_cores(m, n, T, K, N):  # noqa: F811
    assert splits(m, T, K, N) == n
    exact(m, T, K, N, K + T)
