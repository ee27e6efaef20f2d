"""The page calls at the sizes where their forms change, against the plain
reference of tests/_paged.py: tables of more than 1024 entries in a call (the
compaction's gather reads the live tables and a third kernel rewrites them),
sequences of more than 256 pages (table rows in several pieces, a freed row
read again), more than 128 named entries (who names a sequence first goes
through global memory) and more than 1024 (the bookkeeping takes several
turns)."""
import numpy as np
import pytest
import torch

from kv_cache_eviction_dropkv_gb300 import _binding as B
from tests.test_gpu_paged import both, fill, flags_of, ints, pair, same_pool, same_state

pytestmark = pytest.mark.gpu


def kept_positions(r, seqs, kept, seed):
    """[layers][n][H][most] positions, per layer and head some of the sequence's, mostly in order."""
    rng = np.random.default_rng(seed)
    idx = np.zeros((r.L, len(seqs), r.H, max(1, max(kept))), dtype=np.int64)
    for i, s in enumerate(seqs):
        n = r.length[s] if 0 <= s < r.S else 0
        m = min(kept[i], n)
        for layer in range(r.L):
            for h in range(r.H):
                pick = rng.permutation(n)[:m]
                idx[layer, i, h, :m] = pick if h == 1 else np.sort(pick)
    return idx


def compact(c, r, seqs, kept, seed):
    idx = kept_positions(r, seqs, kept, seed)
    c.compact(ints(idx.tolist()), ints(kept), ints(seqs))
    r.compact(idx.tolist(), kept, seqs)


@pytest.mark.parametrize("code,d", [("e4m3", 16), ("int8", 8), ("int8", 48)])
def test_long_tables(code, d):
    """Up to 600 pages a sequence, some of them shared: fork, copy, compaction
    and free by the forms that a table with room takes."""
    c, r = pair(seqs=6, Hkv=2, d=d, pages=1400, page=32, max_pages=600, layers=2, code=code, seed=d)
    fill(c, r, [8293, 40, 1000], seed=3)                    # 260, 2 and 32 pages
    both(c, r, "fork", [0, 2], [3, 4])                      # full pages shared, the last one copied
    same_state(c, r)
    both(c, r, "copy", [0], [5])
    same_state(c, r)
    same_pool(c, r)
    assert flags_of(c) == 0
    # two branches that share their pages, a whole sequence and one that keeps nothing
    compact(c, r, [3, 2, 5, 1], [8290, 333, 900, 0], seed=4)
    same_state(c, r)
    same_pool(c, r)
    both(c, r, "free", [3])                                 # a row of more than 256 pages
    same_state(c, r)
    compact(c, r, [0, 4, 2, 5], [5, 999, 333, 33], seed=5)
    same_state(c, r)
    same_pool(c, r)
    assert flags_of(c) == r.flags == 0
    both(c, r, "free", [0, 1, 2, 4, 5])
    assert int(c.refs.abs().sum()) == 0 and c.check() == 0


def test_long_tables_when_pages_run_out_or_positions_do_not_fit():
    c, r = pair(seqs=4, Hkv=1, d=8, pages=300, page=32, max_pages=400, code="e4m3")
    fill(c, r, [8293, 700])                                 # 260 and 22 of 300 pages
    both(c, r, "copy", [1], [2])                            # 22 more than are free
    compact(c, r, [0, 1], [600, 650], seed=1)               # 19 and 21 wanted, 18 free
    same_state(c, r)
    same_pool(c, r)
    assert flags_of(c) == r.flags == B.FLAG_NO_PAGES
    both(c, r, "fork", [0], [3])
    same_state(c, r)
    c.reset_status()
    idx = kept_positions(r, [0, 1], [40, 33], 2)
    bad = idx.copy()
    bad[0, 0, 0, 7], bad[0, 1, 0, 32] = 8293, -1            # flagged, stored as zeros
    c.compact(ints(bad.tolist()), ints([40, 33]), ints([0, 1]))
    r.compact(idx.tolist(), [40, 33], [0, 1])
    same_state(c, r)
    assert flags_of(c) == B.FLAG_BAD_K
    pool = c.k.float()
    assert torch.all(pool[0, c.table[0, 0], 0, 7] == 0) and torch.all(pool[0, c.table[1, 1], 0, 0] == 0)


@pytest.mark.parametrize("n,M", [(200, 5), (200, 40)])
def test_hundreds_of_named_entries(n, M):
    """More entries than are compared in shared memory: shuffled, named twice,
    out of range, sources named as destinations; short and long tables."""
    S = 500
    rng = np.random.default_rng(n + M)
    c, r = pair(seqs=S, Hkv=1, d=8, pages=1500, page=32, max_pages=M, code="int8", seed=M)
    who = [int(x) for x in rng.permutation(S)[:n]]
    who[17], who[150], who[199] = who[3], who[151], who[40]     # (the later of each is left out)
    who[60], who[130] = S, -1
    new = [int(rng.integers(0, 71)) for _ in who]
    both(c, r, "reserve", new, seqs=who)
    same_state(c, r)
    assert flags_of(c) == r.flags == B.FLAG_BAD_SEQ
    named = [s for i, s in enumerate(who) if 0 <= s < S and s not in who[:i]]
    for part in (named[:100], named[100:]):
        lengths = [r.length[s] for s in part]
        k, v = (torch.randn(len(part), 1, 70, 8, generator=torch.Generator().manual_seed(j)).bfloat16() for j in (1, 2))
        both(c, r, "store", 0, k, v, lengths, seqs=part)
    same_pool(c, r)
    c.reset_status()
    r.flags = 0
    empty = [s for s in range(S) if r.length[s] == 0]
    src = [named[int(rng.integers(0, len(named)))] for _ in range(n)]
    dst = [int(x) for x in rng.permutation(empty)[:n]]
    dst[5], dst[180] = dst[170], dst[179]                       # named twice
    dst[33], src[77], dst[101], src[140] = src[20], S + 7, -1, -3   # a source; out of range
    src[160] = dst[161]                                         # an empty source that is a destination
    both(c, r, "fork", src, dst)
    same_state(c, r)
    same_pool(c, r)
    assert flags_of(c) == r.flags == B.FLAG_BAD_SEQ
    some = [int(x) for x in rng.permutation([s for s in range(S) if r.length[s] > 0])[:n]]
    some += [some[0]] * (n - len(some))
    some[9], some[190] = some[8], S
    compact(c, r, some, [int(rng.integers(0, r.length[s] + 1)) if s < S else 1 for s in some], seed=7)
    same_state(c, r)
    same_pool(c, r)
    assert flags_of(c) == r.flags


def test_over_a_thousand_entries():
    """More entries than the bookkeeping's threads."""
    S, n = 2600, 1300
    rng = np.random.default_rng(1)
    c, r = pair(seqs=S, Hkv=1, d=8, pages=5200, page=32, max_pages=2, code="e4m3")
    lengths = [int(rng.integers(0, 65)) for _ in range(n)]
    both(c, r, "reserve", lengths)                              # sequences 0 .. n - 1, not named
    same_state(c, r)
    k, v = (torch.randn(n, 1, 64, 8, generator=torch.Generator().manual_seed(j)).bfloat16() for j in (1, 2))
    both(c, r, "store", 0, k, v, lengths)
    src = [int(rng.integers(0, n)) for _ in range(n)]
    dst = [int(x) for x in n + rng.permutation(n)]
    dst[1200], dst[1100] = dst[10], src[1250]                   # named twice; a source
    both(c, r, "fork", src, dst)
    same_state(c, r)
    assert flags_of(c) == r.flags == B.FLAG_BAD_SEQ
    some = [int(x) for x in rng.permutation(S)[:n]]
    some[1290] = some[7]
    both(c, r, "reserve", [1 if r.length[s] < 64 else 0 for s in some], seqs=some)
    same_state(c, r)
    compact(c, r, some, [r.length[s] // 2 for s in some], seed=2)
    same_state(c, r)
    same_pool(c, r)
    both(c, r, "copy", [s for s in range(n)][:n], [S] * n)      # out of range, every one
    c.reset_status()
    r.flags = 0
    both(c, r, "reserve", [64] * n, seqs=some)                  # past max_pages, where anything is held
    same_state(c, r)
    assert flags_of(c) == r.flags
    c.free(ints(list(range(S))))
    assert int(c.refs.abs().sum()) == 0
