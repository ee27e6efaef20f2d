"""Attention over shared pages where its references move, where page scales are
far apart and where one chain is long: the shared half's own limits."""
import math

import pytest
import torch

from kv_cache_eviction_dropkv_gb300 import PagedCache
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


def weighted(c, q, seqs):
    """Outputs in 64 bits; sum_j p_j |v_j| of each channel; the largest p_j times V scale."""
    n, Hq, T, d = q.shape
    out, size = (torch.zeros(n, Hq, T, d, dtype=torch.float64, device=DEV) for _ in range(2))
    most = torch.zeros(n, Hq, T, 1, dtype=torch.float64, device=DEV)
    for i, s in enumerate(seqs):
        L = int(c.length[s])
        pages = c.table[s, :-(-L // c.page)].long()
        k, v, scale = ((x.double() * sc[0][pages].double()[..., None, None]).transpose(0, 1).reshape(c.Hkv, -1, x.shape[-1])[:, :L]
                       for x, sc in ((c.k[0].view(torch.uint8)[pages].view(c.k.dtype), c.k_scale),
                                     (c.v[0].view(torch.uint8)[pages].view(c.v.dtype), c.v_scale),
                                     (torch.ones(len(pages), c.Hkv, c.page, 1, device=DEV), c.v_scale)))
        for t in range(T):
            x = q[i, :, t].double().reshape(c.Hkv, -1, d) @ k.transpose(-1, -2) / math.sqrt(d)
            p = torch.softmax(x[..., :L - T + t + 1], -1)
            out[i, :, t], size[i, :, t] = ((p @ y[:, :L - T + t + 1]).reshape(Hq, d) for y in (v, v.abs()))
            most[i, :, t] = (p * scale[:, :L - T + t + 1].transpose(-1, -2)).amax(-1).reshape(Hq, 1)
    return out, size, most


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("d,page,g,T", [(128, 64, 4, 1), (64, 32, 4, 1), (96, 64, 8, 9)])
@pytest.mark.parametrize("rise", [20, 35, 50, 60, 70, 100])
def test_pages_of_tiny_values_behind_one_of_plain_ones(code, d, page, g, T, rise):
    """V scales 2^0 on the first page and 2^-100 on the others, whose keys are
    2^rise times as likely: what the first page's tokens weigh in the outputs
    stands against values 2^100 smaller, so the bound goes by the outputs.

    Bound, W = sum p |v|: 2^-8 of the output (bf16); of W, 2^-11 (P in fp16),
    2^-12 (base-2 logits up to 2^7 in fp32: three roundings, 2^-24 2^7 ln 2
    each, and S) and 2^-23 for each of n tokens' additions; what fp16 drops of
    P, 2^-28 of the row's largest p times V scale for each token, whose code is
    448 (int8: 127) at most."""
    c, seqs, _ = forked([1280], [[1 + i % 5 for i in range(32)]], 8, g, d, page, code, T, seed=d)
    pages = c.table[0, :1280 // page].long()
    first = int(pages[0])
    levels(c, pages, [1.0] + [1.0 + rise] * (len(pages) - 1), 1)
    c.v_scale *= 2.0 ** -100
    c.v_scale[0, first] *= 2.0 ** 100
    q = slopes(32, 8 * g, T, d, 3)
    out = torch.full_like(q, 7.0)
    c.shared_attention(0, q, out, ints(range(0, 33, 2)), seqs=ints(seqs), least=0)
    want, size, most = weighted(c, q, seqs)
    n = int(c.length.max())
    bound = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -12 + n * 2.0 ** -23) * size + n * 2.0 ** -28 * 448 * most
    err = (out.double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    assert c.check() == 0


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("Hq", [8, 72])
@pytest.mark.parametrize("first", [True, False])
def test_a_flat_tail_behind_dominant_keys(code, Hq, first):
    """2^20 shared tokens whose weight is 2^-27.6 of two dominant ones' each,
    0.0025 of the output together, where a CTA has whole units: of 16 rows (the
    two groups take the tiles in turn, a dominant key each) and of 144.

    All values are 1 but the dominant ones', which are 0.  Bound: the bf16
    rounding 2^-8 o; the fp32 sums, every addition off by a last place of a sum
    that only grows: 2^16 products of 16 tokens into an accumulator (2^-23 each
    if it truncates, 2^-7 o), 2^15 blocks into the sum of weights (2^-24 each,
    2^-9 o); 2^-10 o for the exponentials' fp32 arguments; the probabilities'
    fp16 rounding, 2^-32 of the largest for each."""
    tokens, groups = 1 << 20, 2 * torch.cuda.get_device_properties(0).multi_processor_count
    n = 2 * groups
    c = PagedCache(n, 1, 8, 9000, 128, tokens // 128, 1, code, Hq=Hq, device=DEV, groups=groups)
    c.reserve(ints([tokens]))
    at = [0, 128] if first else [tokens - 129, tokens - 1]
    k, v = torch.zeros(1, 1, tokens, 8, dtype=torch.bfloat16), torch.ones(1, 1, tokens, 8, dtype=torch.bfloat16)
    k[..., 1] = 1.0
    k[0, 0, at, 0], k[0, 0, at, 1] = 26.0, 0.0
    v[0, 0, at] = 0.0
    c.store(0, k.to(DEV), v.to(DEV))
    q = torch.zeros(n, Hq, 1, 8, dtype=torch.bfloat16, device=DEV)
    q[..., 0], q[..., 1] = 2.125, 1.0625
    out = torch.zeros_like(q)
    c.shared_attention(0, q, out, ints(range(0, n + 1, 2)), seqs=ints([0] * n), least=0)
    assert c.check() == 0
    pages = c.table[0].long()
    held, ones = ((x[0].view(torch.uint8)[pages].view(x.dtype).double() * s[0][pages].double()[..., None, None])
                  .reshape(tokens, 8) for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)))
    p = torch.softmax(held @ q[0, 0, 0].double() / math.sqrt(8.0), 0)
    want = float((p @ ones)[0])
    assert 0.002 < want < 0.003
    err = float((out.double() - want).abs().max())
    assert err <= (2.0 ** -8 + 2.0 ** -7 + 2.0 ** -9 + 2.0 ** -10) * want + tokens * 2.0 ** -32 * float(p.max()), (err, want)
