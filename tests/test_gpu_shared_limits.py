"""Attention over shared pages where its references move, where page scales are
far apart and where one chain is long: the shared half's own limits."""
import math

import pytest
import torch

from tests.test_gpu_paged import DEV, ints
from tests.test_gpu_shared import check, forked, queries

gpu = pytest.mark.gpu
pytestmark = gpu


def levels(c, pages, bits, seed):
    """Keys of `pages` (sequence order) whose base-2 logits are q[0] bits[i]
    for the i-th page, and a little that tells the tokens apart."""
    g = torch.Generator().manual_seed(seed)
    k = torch.randint(-1, 2, (len(pages), c.Hkv, c.page, c.d), generator=g).float()
    k[..., 0] = 8.0
    c.k.view(torch.uint8)[0, pages] = k.to(c.k.dtype).view(torch.uint8).to(DEV)
    scale = torch.as_tensor(bits, dtype=torch.float64) * math.sqrt(c.d) * math.log(2.0) / 8.0
    c.k_scale[0, pages] = scale.float().to(DEV)[:, None].expand(-1, c.Hkv)


def slopes(n, Hq, T, d, seed):
    """Queries whose first channel is one of a few factors, by row, and small elsewhere."""
    q = queries(n, Hq, T, d, seed) / 64
    f = torch.tensor([1.0, 0.75, 0.5, -1.0, 0.25, 0.875, 0.625], device=DEV)
    q[..., 0] = f[torch.arange(n * Hq * T, device=DEV) % 7].reshape(n, Hq, T)
    return q


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("d,page,g,T", [(128, 64, 4, 1), (64, 32, 4, 1), (96, 64, 8, 9), (128, 32, 8, 9), (64, 64, 8, 9)])
def test_logits_that_rise_in_every_half_tile(code, d, page, g, T):
    """The references move in both halves of a tile and in the next one again:
    outputs and the first half of P are scaled right behind their stores.
    128 units of 8 rows (the two groups take turns) and of 144 (both take every
    tile), 8 tiles and more to a CTA."""
    c, seqs, _ = forked([1280], [[1 + i % 5 for i in range(32)]], 8, g, d, page, code, T, seed=d)
    pages = c.table[0, :1280 // page].long()
    half = torch.arange(len(pages)) * page // 64
    levels(c, pages, 10.0 * (half + 1), 1)
    q = slopes(32, 8 * g, T, d, 3)
    check(c, q, seqs, list(range(0, 33, 2)))
    levels(c, pages, 10.0 * (half + 1) + 4.0 * (half % 3), 1)
    check(c, q, seqs, list(range(0, 33, 2)))
    assert c.check() == 0
