"""Attention of forked sequences over the pages they share, against the
definition in 64 bits and against the call that does not share.

The bound is that of tests/test_gpu_paged.py: the same roundings happen to the
shared tokens (codes and queries exact in fp16, probabilities off by 2^-11 or
2^-32 of the row's largest, fp32 sums, the output rounded to bf16)."""
import math

import pytest
import torch

from kv_cache_eviction_dropkv_gb300 import DropKVError, PagedCache, _binding as B
from tests.test_gpu_paged import DEV, draw_rows, flags_of, ints

gpu = pytest.mark.gpu
pytestmark = gpu


def noise(cache, seed):
    """A pool of random bytes, as after some serving (not-a-number codes among them)."""
    g = torch.Generator().manual_seed(seed)
    for pool, scales in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        pool.view(torch.uint8).copy_(torch.randint(0, 256, pool.shape, generator=g, dtype=torch.uint8))
        scales.copy_(2.0 ** torch.randint(-9, 9, scales.shape, generator=g).float())


def put(cache, seqs, counts, seed, spread=0.5):
    """counts[i] more tokens of sequence seqs[i], in every layer."""
    cache.reserve(ints(counts), seqs=ints(seqs))
    rows = max(1, max(counts))
    for layer in range(cache.layers):
        k, v = (draw_rows(len(seqs), cache.Hkv, rows, cache.d, seed + 10 * layer + j, spread).to(DEV) for j in range(2))
        cache.store(layer, k, v, ints(counts), seqs=ints(seqs))


def forked(prefixes, members, Hkv, g, d, page, code="e4m3", T=1, layers=1, seed=0, spread=0.5):
    """A cache with a sequence per prefix and its forks: members[j] lists the
    own tokens of each fork of prefix j.  Returns it, the forks' numbers in
    groups' order and the groups' starts."""
    roots, n = len(prefixes), sum(len(m) for m in members)
    longest = max(p + max(m + [0]) for p, m in zip(prefixes, members))
    max_pages = -(-longest // page) + 1
    pages = sum(-(-p // page) for p in prefixes) + sum(-(-(p % page + x) // page) + 1 for p, m in zip(prefixes, members) for x in m) + 4
    c = PagedCache(roots + n, Hkv, d, pages, page, max_pages, layers, code, Hq=Hkv * g, T=T, device=DEV, groups=max(1, n))
    noise(c, seed)
    put(c, list(range(roots)), prefixes, seed + 1, spread)
    seqs, starts = [], [0]
    for j, m in enumerate(members):
        mine = list(range(roots + len(seqs), roots + len(seqs) + len(m)))
        if mine:
            c.fork(ints([j] * len(mine)), ints(mine))
        seqs += mine
        starts.append(len(seqs))
    put(c, seqs, [x for m in members for x in m], seed + 2, spread)
    assert c.check() == 0
    return c, seqs, starts


def definition(c, q, seqs, layer=0):
    """Outputs in 64 bits and the largest |v| a row sees."""
    n, Hq, T, d = q.shape
    out = torch.zeros(n, Hq, T, d, dtype=torch.float64, device=DEV)
    vmax = torch.zeros(n, Hq, T, dtype=torch.float64, device=DEV)
    for i, s in enumerate(seqs):
        if not 0 <= s < c.seqs:
            continue
        L = int(c.length[s])
        pages = c.table[s, :-(-L // c.page)].long()
        k, v = ((x[layer].view(torch.uint8)[pages].view(x.dtype).double() * sc[layer][pages].double()[..., None, None])
                .transpose(0, 1).reshape(c.Hkv, -1, d)[:, :L] for x, sc in ((c.k, c.k_scale), (c.v, c.v_scale)))
        for t in range(T):
            p = L - T + t
            if p >= 0:
                x = q[i, :, t].double().reshape(c.Hkv, -1, d) @ k[:, :p + 1].transpose(-1, -2) / math.sqrt(d)
                out[i, :, t] = (torch.softmax(x, -1) @ v[:, :p + 1]).reshape(Hq, d)
                vmax[i, :, t] = v[:, :p + 1].abs().amax((1, 2)).repeat_interleave(Hq // c.Hkv)
    return out, vmax


def check(c, q, seqs, starts, layer=0):
    out = torch.full_like(q, 7.0)
    c.shared_attention(layer, q, out, ints(starts), seqs=ints(seqs), least=0)
    want, vmax = definition(c, q, seqs, layer)
    n = int(c.length.max())
    err = (out.double() - want).abs()
    bound = 1.125 * (2.0 ** -8 * want.abs() + (2.0 ** -10 + n * 2.0 ** -25) * vmax[..., None])
    assert bool((err <= bound).all()), float((err / bound.clamp_min(1e-300)).max())
    return out


def queries(n, Hq, T, d, seed):
    return draw_rows(n, Hq, T, d, seed, 0.3).to(DEV)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("page,d,Hkv,g,T", [(32, 8, 3, 2, 1), (32, 96, 1, 7, 2), (64, 40, 2, 1, 3), (64, 128, 2, 4, 1),
                                            (128, 72, 1, 3, 1), (128, 128, 2, 8, 2), (64, 64, 2, 4, 1), (32, 16, 1, 1, 5)])
def test_one_group(code, page, d, Hkv, g, T):
    c, seqs, starts = forked([5 * page + 3], [[1, 2, page, 40, 7]], Hkv, g, d, page, code, T, seed=d)
    check(c, queries(5, Hkv * g, T, d, 3), seqs, starts)
    assert c.check() == 0


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [8, 16, 24, 48, 56, 80, 88, 104, 112, 120])
def test_head_widths(code, d):
    """Codes in pieces of 8 and 16, in each of the three tile widths; the last tile half full."""
    c, seqs, starts = forked([3 * 128 + 64 + 5], [[1, 70, 33]], 2, 3, d, 64, code, seed=d)
    check(c, queries(3, 6, 1, d, 3), seqs, starts)
    assert c.check() == 0


@pytest.mark.parametrize("prefix", [0, 1, 31, 32, 33, 127, 128, 129, 255, 256, 300, 4000])
def test_prefix_lengths(prefix):
    """Nothing shared, parts of tiles, whole ones; three rows, of which the first may see one token less than a page."""
    for T, own in ((1, [0, 1, 5]), (3, [3, 4, 64])):
        c, seqs, starts = forked([prefix], [[x + (prefix == 0) for x in own]], 2, 2, 64, 32, T=T, seed=prefix)
        check(c, queries(3, 4, T, 64, 3), seqs, starts)
        assert c.check() == 0


@pytest.mark.parametrize("rows", [16, 17, 32, 33, 40, 70])
def test_more_rows_than_a_tile(rows):
    """128, 136, 256, 264, 320, 560 rows of a KV head: units of 128 and 256 rows, the last one short."""
    c, seqs, starts = forked([700], [[1 + (5 * i) % 50 for i in range(rows)]], 2, 8, 128, 64, seed=rows)
    check(c, queries(rows, 16, 1, 128, 3), seqs, starts)
    assert c.check() == 0


def test_many_groups_of_all_sizes():
    """Groups of no, one, few and many members, prefixes from nothing to 3000
    tokens, more units than processors: runs that cross units of both widths."""
    sizes = [3, 0, 1, 40, 2, 0, 7, 1, 20, 5]
    prefixes = [3000, 64, 500, 777, 31, 100, 1281, 2000, 130, 65]
    members = [[(11 * j + 7 * i) % 90 + 1 for i in range(m)] for j, m in enumerate(sizes)]
    for Hkv, g, d, page in ((16, 4, 64, 32), (3, 8, 96, 64)):
        c, seqs, starts = forked(prefixes, members, Hkv, g, d, page, seed=d)
        check(c, queries(len(seqs), Hkv * g, 1, d, 3), seqs, starts)
        assert c.check() == 0


@pytest.mark.parametrize("code,d", [("e4m3", 128), ("int8", 64)])
def test_short_segments(code, d):
    """Units of one to three tiles, so that runs hold several and the two
    groups of warps take turns at odd counts."""
    for prefix in (128, 256, 384, 200):
        members = [[1 + (i + j) % 9 for i in range(2 + j % 3)] for j in range(24)]
        c, seqs, starts = forked([prefix + 32 * (j % 2) for j in range(24)], members, 16, 2, d, 32, code, seed=prefix)
        check(c, queries(len(seqs), 32, 1, d, 3), seqs, starts)
        assert c.check() == 0


def test_long_prefix_and_long_own_tokens():
    c, seqs, starts = forked([40000], [[1, 3000, 20, 9000]], 2, 4, 128, 64, seed=1)
    check(c, queries(4, 8, 1, 128, 3), seqs, starts)
    c, seqs, starts = forked([20000], [[100 + i for i in range(40)]], 1, 8, 64, 128, "int8", seed=2)
    check(c, queries(40, 8, 1, 64, 3), seqs, starts)


def test_loud_tokens_and_pages_of_very_different_scales():
    """References move late, V scales differ by 2^40 from page to page, a dominant key in the last shared page."""
    c, seqs, starts = forked([1000], [[5, 40, 33]], 2, 4, 64, 32, seed=4, spread=1.0)
    q = queries(3, 8, 1, 64, 5)
    shared = c.table[seqs[0], :1000 // 32].long()
    c.v_scale[0, shared] *= torch.exp2(torch.linspace(-30, 10, len(shared), device=DEV).round())[:, None]
    check(c, q, seqs, starts)
    c.k_scale[0, shared[-1]] *= 4.0
    check(c, q, seqs, starts)
    c.v_scale[0, shared] = 2.0 ** -120
    check(c, q, seqs, starts)
    assert c.check() == 0


def test_layers_orders_and_what_is_not_shared():
    c, seqs, starts = forked([300, 200], [[5, 9, 1], [4, 8]], 2, 2, 64, 32, layers=2, seed=7)
    q = queries(5, 4, 1, 64, 3)
    check(c, q, seqs, starts, layer=1)
    # members in another order, one of them twice, groups across the two prefixes: nothing is shared, the results stand
    check(c, q, [seqs[i] for i in (2, 0, 1, 4, 3)], starts)
    check(c, q, [seqs[0], seqs[0], seqs[1], seqs[3], seqs[3]], starts)
    check(c, q, seqs, [0, 5])
    check(c, q, seqs, [0, 1, 2, 3, 4, 5])
    check(c, q, [0, seqs[0], seqs[1], 1, seqs[3]], starts)          # with the roots themselves
    # a copy shares no page
    fresh = PagedCache(6, 2, 64, 80, 32, 12, Hq=4, groups=2, device=DEV)
    noise(fresh, 1)
    put(fresh, [0], [300], 3)
    fresh.copy(ints([0]), ints([1]))
    fresh.fork(ints([0, 0]), ints([2, 3]))
    check(fresh, q[:3], [1, 2, 3], [0, 3])
    check(fresh, q[:3], [2, 3, 0], [0, 2, 3])
    assert c.check() == 0 and fresh.check() == 0


def test_members_that_take_no_part():
    """Empty, short, missing sequences among the members: the others share, these get what attention() gives."""
    c, seqs, starts = forked([500], [[5, 9, 1, 40]], 2, 4, 64, 64, T=2, seed=9)
    short = PagedCache(8, 2, 64, 60, 64, 12, Hq=8, T=2, groups=3, device=DEV)
    noise(short, 3)
    put(short, [0, 1], [500, 30], 5)
    short.fork(ints([0, 0, 0]), ints([2, 3, 4]))
    put(short, [2, 3, 4], [3, 1, 20], 6)
    q = queries(7, 8, 2, 64, 3)
    for members in ([5, 2, 3, 1, 4, 6, 5], [1, 1, 2, 5, 5, 3, 4], [5, 5, 5, 5, 5, 5, 2]):
        check(short, q, members, [0, 7])
    assert short.check() == 0
    out = check(short, q, [2, -1, 3, 8, 4, 1, 5], [0, 7])
    assert flags_of(short) == B.FLAG_BAD_SEQ
    assert not out[1].any() and not out[3].any() and not out[6].any()


def test_flags_and_refusals():
    c, seqs, starts = forked([200], [[5, 9, 1, 40]], 2, 2, 64, 32, seed=9)
    q = queries(4, 4, 1, 64, 3)
    for bad in ([1, 4], [0, 3], [0, 3, 2, 4], [0, 5], [0, -1, 4], [4, 4]):
        out = torch.full_like(q, 7.0)
        c.shared_attention(0, q, out, ints(bad), seqs=ints(seqs), least=0)
        assert flags_of(c) == B.FLAG_BAD_LENGTH
        c.reset_status()
        plain = torch.empty_like(q)
        c.attention(0, q, plain, seqs=ints(seqs))
        assert float((out.double() - plain.double()).abs().max()) <= 2.0 ** -7 * float(plain.abs().max())
    # a table entry that is no page is not shared, and flagged where it is read
    kept = c.table.clone()
    c.table[seqs[1], 3] = -1
    out = torch.empty_like(q)
    c.shared_attention(0, q, out, ints(starts), seqs=ints(seqs), least=0)
    assert flags_of(c) == B.FLAG_BAD_PAGE
    c.table[seqs, 2] = c.pages
    c.shared_attention(0, q, out, ints(starts), seqs=ints(seqs), least=0)
    assert flags_of(c) == B.FLAG_BAD_PAGE
    c.table.copy_(kept)
    c.reset_status()
    for bad in (dict(q=q.float()), dict(out=out[:2]), dict(groups=torch.zeros(2, device=DEV)), dict(layer=1), dict(seqs=ints([1])),
                dict(q=torch.cat((q, q), 2), out=torch.cat((q, q), 2)), dict(groups=ints(list(range(7))))):
        with pytest.raises(ValueError):
            c.shared_attention(**{**dict(layer=0, q=q, out=out, groups=ints(starts), seqs=ints(seqs)), **bad})
    with pytest.raises(DropKVError):
        c.shared_attention(0, q, q, ints(starts), seqs=ints(seqs))
    with pytest.raises(DropKVError):
        c.shared_attention(0, q, out, ints([0]), seqs=ints(seqs))
    c.shared_attention(0, q[:0], out[:0], ints([0, 0]), seqs=ints([]))
    assert c.check() == 0


def test_small_calls_are_attention():
    """Below `least` bytes the call is attention(), bit by bit."""
    c, seqs, starts = forked([200], [[5, 9, 1, 40]], 2, 2, 64, 32, seed=9)
    q = queries(4, 4, 1, 64, 3)
    plain, out = torch.empty_like(q), torch.empty_like(q)
    c.attention(0, q, plain, seqs=ints(seqs))
    most = 2 * 4 * c.max_pages * 32 * 2 * 64
    for least in (-1, most + 1):
        c.shared_attention(0, q, out.fill_(7.0), ints(starts), seqs=ints(seqs), least=least)
        assert torch.equal(out, plain)
    c.shared_attention(0, q, out.fill_(7.0), ints([1, 2]), seqs=ints(seqs))     # (not looked at)
    assert torch.equal(out, plain) and c.check() == 0
    c.shared_attention(0, q, out, ints([1, 2]), seqs=ints(seqs), least=most)
    assert flags_of(c) == B.FLAG_BAD_LENGTH


def test_groups_of_one_are_attention():
    """Where sharing saves nothing the call is attention(), however much there is to read."""
    n = 8
    c = PagedCache(n + 1, 2, 64, 40, 128, 8192, 1, "e4m3", Hq=8, T=1, device=DEV, groups=n)
    seqs = list(range(1, n + 1))
    put(c, [0], [300], 3)
    c.fork(ints([0] * n), ints(seqs))
    put(c, seqs, [1 + 7 * i for i in range(n)], 4)
    assert c.check() == 0
    q = queries(n, 8, 1, 64, 5)
    plain, out = torch.empty_like(q), torch.empty_like(q)
    c.attention(0, q, plain, seqs=ints(seqs))
    c.shared_attention(0, q, out.fill_(7.0), ints([1] * (n + 1)), seqs=ints(seqs))     # (not looked at)
    assert torch.equal(out, plain) and c.check() == 0
    c.shared_attention(0, q, out, ints([0, n - 1]), seqs=ints(seqs))
    assert flags_of(c) == B.FLAG_BAD_LENGTH


def test_not_a_number_codes_reach_their_rows_only():
    c, seqs, starts = forked([200, 200], [[5, 9], [1, 40]], 2, 2, 64, 32, seed=9)
    q = queries(4, 4, 1, 64, 3)
    good = check(c, q, seqs, starts)
    for pool in (c.k, c.v):
        pg = int(c.table[seqs[0], 1])
        was = pool.view(torch.uint8)[0, pg, 1, 3, 5].clone()
        pool.view(torch.uint8)[0, pg, 1, 3, 5] = 0x7F
        out = torch.empty_like(q)
        c.shared_attention(0, q, out, ints(starts), seqs=ints(seqs), least=0)
        pool.view(torch.uint8)[0, pg, 1, 3, 5] = was
        assert torch.equal(out[2:], good[2:]) and torch.equal(out[:, :2], good[:, :2])
        assert bool(out[:2, 2:].isnan().any(-1).all())


def test_two_captured_calls_and_other_streams():
    """Replayed graphs follow the cache as it grows and as its branches change; two calls in a row share the workspace."""
    c, seqs, starts = forked([700, 90], [[5, 9, 30, 2], [1, 40]], 2, 4, 128, 64, layers=2, seed=11)
    q = queries(6, 8, 1, 128, 3)
    members, groups = ints(seqs), ints(starts)
    outs = [torch.zeros_like(q) for _ in range(2)]

    def step():
        for layer in range(2):
            c.shared_attention(layer, q, outs[layer], groups, seqs=members, least=0)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for grow in range(3):
        put(c, seqs, [(7 * grow + i) % 5 + 1 for i in range(6)], 50 + grow)
        if grow == 2:                         # other tables: the groups swap members
            members.copy_(ints([seqs[4], seqs[5], seqs[0], seqs[1], seqs[2], seqs[3]]))
            groups.copy_(ints([0, 2, 6]))
        graph.replay()
        torch.cuda.synchronize()
        for layer in range(2):
            want = check(c, q, members.tolist(), groups.tolist(), layer)
            assert torch.equal(outs[layer], want)
    assert c.check() == 0


def test_more_entries_than_one_cta_plans():
    """1300 entries: the groups stand in global memory."""
    sizes = [400, 1, 0, 500, 3, 396]
    c, seqs, starts = forked([130, 64, 32, 257, 40, 96], [[1 + (i + j) % 5 for i in range(m)] for j, m in enumerate(sizes)],
                             1, 2, 16, 32, seed=5)
    q = queries(len(seqs), 2, 1, 16, 3)
    check(c, q, seqs, starts)
    c.table[seqs[3], 1] = c.table[seqs[1000], 0]                 # one member of the first group differs in its second page
    check(c, q, seqs, starts)
    assert c.check() == 0
    c.shared_attention(0, q, torch.empty_like(q), ints([0, 1299]), seqs=ints(seqs), least=0)
    assert flags_of(c) == B.FLAG_BAD_LENGTH


def test_offsets_past_32_bits():
    """Pages whose codes lie more than 2^32 bytes into the pool: shared, read back and stored to."""
    from kv_cache_eviction_dropkv_gb300 import Rotary

    c = PagedCache(4, 8, 128, 36000, 128, 24, 1, "e4m3", Hq=16, T=1, device=DEV, groups=1)
    c.refs[:35900] = 1                                          # the free pages are the last ones
    assert 35900 * 8 * 128 * 128 > 2 ** 32
    put(c, [0], [2000], 3)
    c.fork(ints([0, 0, 0]), ints([1, 2, 3]))
    put(c, [1, 2, 3], [5, 200, 40], 7)
    assert int(c.table[1, 0]) >= 35900
    check(c, queries(3, 16, 1, 128, 3), [1, 2, 3], [0, 3])
    k, v, q = (draw_rows(3, h, 4, 128, 9 + h).to(DEV) for h in (8, 8, 16))
    c.reserve(ints([4, 4, 4]), seqs=ints([1, 2, 3]))
    plan, q_out = Rotary(128, dims=0, device=DEV), torch.empty_like(q)
    c.store_rotated(0, plan, q, k, v, q_out, seqs=ints([1, 2, 3]))
    assert torch.equal(q_out, q)
    got = [torch.empty_like(k) for _ in range(2)]
    c.read(0, *got, starts=c.length[1:] - 4, seqs=ints([1, 2, 3]))
    for a, b in zip(got, (k, v)):                               # e4m3: half a step of four bits, or of the smallest number
        scale = torch.maximum(c.k_scale.max(), c.v_scale.max()).item()
        assert bool(((a.double() - b.double()).abs() <= 2.0 ** -4 * b.double().abs() + 2.0 ** -10 * scale).all())
    assert c.check() == 0
