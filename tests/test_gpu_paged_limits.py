"""The paged 8-bit cache at the ends of its ranges, against the plain reference
of tests/_paged.py or the formulas themselves."""
import numpy as np
import pytest
import torch

from kv_cache_eviction_dropkv_gb300 import PagedCache
from tests.test_gpu_paged import DEV, draw_rows, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page,rows", [(128, 200), (32, 200), (64, 4096)])
def test_store_behind_the_longest_sequence_touches_nothing_else(page, rows):
    """A sequence as long as lengths go, more rows than are stored: the pages
    that `rows` tokens could touch end behind the last one a 32-bit count
    reaches, and there lies the table row of the next sequence.  (All but its
    last pages are one page: a store looks at those that it writes.)"""
    M = (1 << 31) // page - 1
    c = PagedCache(2, 1, 8, 40, page, M, 1, device=DEV)
    c.table[0] = 0
    c.table[0, M - 1] = 1
    c.table[1, :32] = ints(list(range(2, 34)))
    c.count.copy_(ints([M, 32]))
    c.length.copy_(ints([M * page, 32 * page]))
    c.refs[:34] = 1
    c.k_scale.fill_(0.25)
    c.v_scale.fill_(0.5)
    c.k.view(torch.uint8).fill_(0x38)                       # ones
    c.v.view(torch.uint8).fill_(0x38)
    want = [t.clone() for t in (c.k.float(), c.v.float(), c.k_scale, c.v_scale)]
    x = torch.full((1, 1, rows, 8), 2.0, dtype=torch.bfloat16, device=DEV)
    c.store(0, x, x, ints([1]))
    assert c.check() == 0
    want[0][0, 1, 0, page - 1] = 8.0                        # 2 at the scale that the page holds
    want[1][0, 1, 0, page - 1] = 4.0
    for got, w in zip((c.k.float(), c.v.float(), c.k_scale, c.v_scale), want):
        assert torch.equal(got, w)
