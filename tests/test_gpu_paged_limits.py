"""The paged 8-bit cache at the ends of its ranges, against the plain reference
of tests/_paged.py or the formulas themselves."""
import math

import pytest
import torch

from kv_cache_eviction_dropkv_gb300 import PagedCache, _binding as B
from tests.test_gpu_paged import DEV, both, draw_rows, fill, flags_of, ints, pair, same_pool, same_state

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


# ------------------------------------------------------------------ a refused reservation
def same(c, r):
    same_state(c, r)
    same_pool(c, r)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_what_was_granted_is_what_is_stored(code):
    """Steps whose reservation is refused, wholly or for some entries, store
    nothing in their place: the tokens before them stay as they were."""
    c, r = pair(seqs=4, pages=9, max_pages=4, code=code)
    fill(c, r, [64, 33, 1, 128], seed=2)                    # 2, 2, 1 and 4 pages: all
    k, v = (draw_rows(4, 2, 3, 64, 7 + j) for j in range(2))

    def step(extra, want, seqs=None):
        got = ints([9] * len(extra))
        before = list(r.length)
        c.reserve(ints(extra), granted=got, seqs=None if seqs is None else ints(seqs))
        r.reserve(extra, seqs)
        assert got.tolist() == want
        who = list(range(len(extra))) if seqs is None else seqs
        assert [r.length[s] - before[s] if s not in who[:i] else 0 for i, s in enumerate(who)] == want
        n = len(extra)
        c.store(0, k[:n].to(DEV), v[:n].to(DEV), got, seqs=None if seqs is None else ints(seqs))
        r.store(0, k[:n].float().numpy(), v[:n].float().numpy(), want, seqs)
        same(c, r)

    step([1, 1, 1, 0], [0, 0, 0, 0])                        # a page too few: nothing for anybody
    assert flags_of(c) == r.flags == B.FLAG_NO_PAGES
    both(c, r, "free", [2])
    step([1, 3, 0, 1], [1, 3, 0, 0])                        # past max_pages: that entry alone
    assert flags_of(c) == r.flags == B.FLAG_NO_PAGES | B.FLAG_OVERFLOW
    step([2, -1, 2], [2, 0, 0], seqs=[1, 0, 1])             # negative; named twice
    assert flags_of(c) == r.flags
    step([2, 1 << 30], [2, 0], seqs=[0, 1])
    assert flags_of(c) == r.flags


def test_captured_steps_stop_where_pages_run_out():
    """A captured decode step, replayed past the last page."""
    c, r = pair(seqs=2, Hkv=1, d=16, pages=5, page=32, max_pages=5, Hq=2)
    fill(c, r, [60, 30], seed=5)
    k, v = (draw_rows(2, 1, 1, 16, 7 + j) for j in range(2))
    kd, vd, one, got = k.to(DEV), v.to(DEV), ints([1, 1]), ints([0, 0])

    def step():
        c.reserve(one, granted=got)
        c.store(0, kd, vd, got)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(60):
        graph.replay()
        before = list(r.length)
        r.reserve([1, 1])
        r.store(0, k.float().numpy(), v.float().numpy(), [a - b for a, b in zip(r.length, before)])
    same(c, r)
    assert r.length == [94, 64] and got.tolist() == [0, 0]   # sequence 1 wants the sixth page
    assert flags_of(c) == r.flags == B.FLAG_NO_PAGES


def test_granted_over_a_thousand_entries_and_refusals():
    S = 1300
    c, r = pair(seqs=S, Hkv=1, d=8, pages=S, page=32, max_pages=1)
    extra = [(7 * i) % 40 for i in range(S)]                # over 32: past the table
    got = ints([9] * S)
    c.reserve(ints(extra), granted=got)
    assert got.tolist() == [e if e <= 32 else 0 for e in extra]
    for bad in (got[:5], got.long(), got.cpu(), ints([0, 0] * S)[::2]):
        with pytest.raises(ValueError):
            c.reserve(ints(extra), granted=bad)


# ------------------------------------------------------------------ a long, flat tail
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("first", [True, False])
def test_a_flat_tail_behind_one_dominant_key(code, first):
    """2^20 tokens whose weight is 2^-25.5 of the first (or last) token's each,
    0.022 of the output together, where a warp has a whole sequence to itself.

    All tokens but the dominant one are alike (value 1; the dominant one's is
    0), so o = N w / (1 + N w).  Bound: the bf16 rounding 2^-8 o; the fp32
    sums, every addition off by a last place of a sum that only grows: 2^16
    products of 16 tokens into an accumulator (2^-23 each if it truncates, 2^-7
    o), 2^15 tiles into the sum of weights (2^-24 each, 2^-9 o); 2^-10 o for
    the exponentials' fp32 arguments; the probabilities' fp16 rounding, 2^-32
    each, N 2^-32 together."""
    n, tokens = 2000, 1 << 20                               # more sequences than a wave has warps
    c = PagedCache(n, 1, 8, 9000, 128, tokens // 128, 1, code, device=DEV)
    c.reserve(ints([tokens]))
    at = 0 if first else tokens - 1
    k, v = torch.zeros(1, 1, tokens, 8, dtype=torch.bfloat16), torch.ones(1, 1, tokens, 8, dtype=torch.bfloat16)
    k[0, 0, at, 0] = 26.0                                   # (an e4m3 number)
    v[0, 0, at] = 0.0
    c.store(0, k.to(DEV), v.to(DEV))
    page = int(c.table[0, at // 128])
    held = float(c.k[0, page, 0, at % 128, 0].float() * c.k_scale[0, page, 0])
    ones = c.v[0, int(c.table[0, 100]), 0].double() * c.v_scale[0, int(c.table[0, 100]), 0].double()
    q = torch.zeros(n, 1, 1, 8, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 1.921875
    out = torch.zeros_like(q)
    c.attention(0, q, out, seqs=ints([0] * n))              # every entry reads the one sequence
    assert c.check() == 0
    w = (tokens - 1) * math.exp(-1.921875 * held / math.sqrt(8.0))
    want = float(ones.mean()) * w / (1 + w)
    assert 0.02 < want < 0.025
    err = float((out.double() - want).abs().max())
    assert err <= (2.0 ** -8 + 2.0 ** -7 + 2.0 ** -9 + 2.0 ** -10) * want + tokens * 2.0 ** -32, (err, want)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_attention_over_the_longest_sequence(code):
    """2^31 - 128 tokens, all pages one page: positions at the end of 32 bits.

    Without a window the weights are the page's own, repeated (the last row
    sees every token, the one before all but one of 2^31).  Bound: the tests'
    2^-8 |o| + 2^-10 V, and the fp32 sums over a warp's 2^26 / 912 tiles at
    least: two additions a tile into an accumulator, 2^-23 V each if it
    truncates, one of its sum of weights, 2^-24 |o| each."""
    page, d = 128, 8
    M = (1 << 31) // page - 1
    c = PagedCache(1, 1, d, 2, page, M, 1, code, Hq=2, T=2, device=DEV)
    c.table.zero_()
    c.count.fill_(1)
    c.length.fill_(page)
    c.refs[0] = 1
    k, v = (draw_rows(1, 1, page, d, 3 + i) for i in range(2))
    c.store(0, k.to(DEV), v.to(DEV))
    kk, vv = (x[0, 0, 0].double() * s[0, 0, 0].double() for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)))
    c.count.fill_(M)
    c.length.fill_(M * page)
    q = draw_rows(1, 2, 2, d, 9, spread=0.3).to(DEV)
    out = torch.full_like(q, 7.0)
    c.attention(0, q, out)
    assert c.check() == 0
    x = q[0].double() @ kk.T / math.sqrt(d)                 # [head][row][page slot]
    want, top = torch.softmax(x, -1) @ vv, float(vv.abs().max())
    tiles = (1 << 26) / 912
    bound = (2.0 ** -8 + tiles * 2.0 ** -24) * want.abs() + (2.0 ** -10 + 2 * tiles * 2.0 ** -23) * top
    assert torch.all((out[0].double() - want).abs() <= bound)
    for window, sinks in ((1000, 5), (1, 0), (1, 200), (130, (1 << 31) - 1 if code == "int8" else 64)):
        out.fill_(7.0)
        c.attention(0, q, out, window=window, sinks=sinks)
        assert c.check() == 0
        for t in range(2):
            p = M * page - 2 + t
            seen = list(range(max(0, p - window + 1), p + 1)) if sinks <= 200 else None
            if seen is None:                                # every token is a first token
                w, bd = want[:, t], bound[:, t]
            else:
                j = torch.tensor(list(range(min(sinks, seen[0]))) + seen, device=DEV) % page
                w = torch.softmax(x[:, t][:, j], -1) @ vv[j]
                bd = 1.125 * (2.0 ** -8 * w.abs() + 2.0 ** -10 * top)
            assert torch.all((out[0, :, t].double() - w).abs() <= bd), (window, sinks, t)
