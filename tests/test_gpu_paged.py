"""The paged 8-bit cache on the GPU against the plain reference of
tests/_paged.py: codes, scales and page state exactly, attention within bounds
that count the kernel's roundings.

Attention bound per output element, with a = |o| of the reference, V = the
largest |v| the row sees, n the tokens: the output is rounded to bf16 (2^-8 a);
each probability enters the product as fp16 (2^-11 of itself, so at most
2^-11 V after the division by their sum; below fp16's normal range at most
2^-25 of the largest, n 2^-25 V together); the exponentials' arguments are
fp32 sums of d <= 128 products of fp16 codes and query elements, of which no
test has one above 2^6 in the base-2 scale: their error is below
2^6 * 128 * 2^-24 = 2^-11 in the worst order of summation, again at most
2^-11 V.  Sum: 2^-8 a + (2^-10 + n 2^-25) V; a margin of 1/8 covers the fp32
sums themselves."""
import numpy as np
import pytest
import torch

from kv_cache_eviction_dropkv_gb300 import DropKVError, PagedCache, _binding as B
from tests import _paged as R

gpu = pytest.mark.gpu
pytestmark = gpu
DEV = torch.device("cuda", 0) if torch.cuda.is_available() else None


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def pair(seqs=4, Hkv=2, d=64, pages=24, page=32, max_pages=8, layers=1, code="e4m3", Hq=None, T=1, seed=0):
    """A cache whose pool holds random bytes, and the reference holding the same values."""
    c = PagedCache(seqs, Hkv, d, pages, page, max_pages, layers, code, Hq=Hq, T=T, device=DEV)
    r = R.RefCache(seqs, Hkv, d, pages, page, max_pages, layers, code)
    g = torch.Generator().manual_seed(seed)
    for pool, scales, name in ((c.k, c.k_scale, "k"), (c.v, c.v_scale, "v")):
        raw = torch.randint(0, 256, pool.shape, generator=g, dtype=torch.uint8)
        pool.view(torch.uint8).copy_(raw)
        scales.copy_(2.0 ** torch.randint(-9, 9, scales.shape, generator=g).float())
        setattr(r, name, pool.cpu().double().numpy())
        setattr(r, name + "s", scales.cpu().double().numpy())
    return c, r


def draw_rows(n, Hkv, rows, d, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, Hkv, rows, d, generator=g) * torch.exp(spread * torch.randn(n, Hkv, rows, 1, generator=g))
    return x.bfloat16()


def same_state(c, r):
    assert c.refs.tolist() == r.refs
    assert c.length.tolist() == r.length
    assert c.count.tolist() == [len(t) for t in r.table]
    want = [t + [-1] * (r.M - len(t)) for t in r.table]
    assert c.table.tolist() == want


def same_pool(c, r):
    for pool, scales, want, want_s in ((c.k, c.k_scale, r.k, r.ks), (c.v, c.v_scale, r.v, r.vs)):
        np.testing.assert_array_equal(scales.cpu().double().numpy(), want_s)
        np.testing.assert_array_equal(pool.cpu().double().numpy(), want)


def flags_of(c):
    return int(c.status.item()) & 0xFFFFFFFF


def both(c, r, name, *args, **kw):
    """The same call on the cache (device tensors) and on the reference."""
    def dev(x):
        if isinstance(x, torch.Tensor):
            return x.to(DEV)
        if isinstance(x, list):
            return ints(x)
        return x

    def plain(x):
        return x.float().numpy() if isinstance(x, torch.Tensor) else x

    getattr(c, name)(*[dev(a) for a in args], **{k: dev(v) for k, v in kw.items()})
    getattr(r, "fork" if name == "copy" else name)(*[plain(a) for a in args], **kw,
                                                   **({"share": False} if name == "copy" else {}))


def fill(c, r, lengths, seed=0, spread=1.0, seqs=None):
    both(c, r, "reserve", lengths, seqs=seqs)
    rows = max(1, max(lengths))
    for layer in range(c.layers):
        k = draw_rows(len(lengths), c.Hkv, rows, c.d, seed + 2 * layer, spread)
        v = draw_rows(len(lengths), c.Hkv, rows, c.d, seed + 2 * layer + 1, spread)
        both(c, r, "store", layer, k, v, lengths, seqs=seqs)


def check_attention(c, r, q, layer=0, window=0, sinks=0, seqs=None, out=None):
    qd = q.to(DEV)
    out = torch.full_like(qd, 7.0) if out is None else out
    c.attention(layer, qd, out, window=window, sinks=sinks, seqs=None if seqs is None else ints(seqs))
    ref, vmax = r.attention(layer, q.float().numpy(), window, sinks, seqs)
    n = max(r.length)
    err = np.abs(out.cpu().double().numpy() - ref)
    bound = 1.125 * (2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + n * 2.0 ** -25) * vmax[..., None])
    assert np.all(err <= bound), float((err / np.maximum(bound, 1e-300)).max())
    return out


# ------------------------------------------------------------------ store
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("page,d,Hkv", [(32, 8, 3), (32, 96, 1), (64, 40, 2), (64, 128, 2), (128, 72, 1), (128, 128, 1)])
def test_store_matches_reference(code, page, d, Hkv):
    """Prompts of no, one and many tokens, then single tokens and runs behind
    partly filled pages, whose scale may grow; other slots keep their bytes."""
    c, r = pair(seqs=5, Hkv=Hkv, d=d, pages=30, page=page, max_pages=6, layers=2, code=code, seed=d)
    fill(c, r, [0, 1, page - 1, page, 2 * page + 3], seed=1)
    same_pool(c, r)
    for step in range(4):                     # louder and louder tokens: most scales grow
        new = [[1, 1, 1, 1, 1], [3, 0, 2, page, 1], [1, 2, 0, 1, 40], [1, 1, 1, 1, 1]][step]
        both(c, r, "reserve", new)
        k, v = (draw_rows(5, Hkv, max(new), d, 100 + 10 * step + j) * 2.0 ** (step - 1) for j in range(2))
        both(c, r, "store", step % 2, k, v, new)
    same_state(c, r)
    same_pool(c, r)
    assert c.check() == 0 and r.flags == 0


def test_store_of_the_same_tokens_again_changes_nothing():
    c, r = pair(code="int8", seed=3)
    fill(c, r, [5, 40, 64, 1])
    k, v = (draw_rows(4, 2, 40, 64, 50 + j) for j in range(2))
    c.store(0, k.to(DEV), v.to(DEV), ints([5, 7, 40, 1]))
    before = [t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale)]
    c.store(0, k.to(DEV), v.to(DEV), ints([5, 7, 40, 1]))
    for a, b in zip(before, (c.k, c.v, c.k_scale, c.v_scale)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_store_extreme_values(code):
    """Zeros, the smallest and largest bf16 numbers, ties, infinities and not-a-number."""
    c, r = pair(seqs=2, Hkv=1, d=16, pages=8, page=32, max_pages=4, code=code)
    k, v = torch.zeros(2, 1, 40, 16), torch.zeros(2, 1, 40, 16)
    k[0, 0, 1] = 2.0 ** -133
    k[0, 0, 33] = 3.3e38
    k[1, 0, :, :] = torch.arange(640).reshape(40, 16) / 8.0 + 448.0 / 16       # many ties
    v[0, 0, 0, 0], v[0, 0, 0, 1], v[0, 0, 0, 2] = float("inf"), float("-inf"), float("nan")
    v[0, 0, 1, 3] = 2.5
    v[1, 0, 35] = float("nan")
    both(c, r, "reserve", [40, 40])
    both(c, r, "store", 0, k.bfloat16(), v.bfloat16())
    same_pool(c, r)
    assert flags_of(c) == r.flags == B.FLAG_NONFINITE
    with pytest.raises(DropKVError) as e:
        c.check()
    assert e.value.code == 4


def test_store_refusals_on_the_device():
    c, r = pair()
    fill(c, r, [33, 40, 0, 0])
    k, v = (draw_rows(4, 2, 8, 64, 9 + j) for j in range(2))
    both(c, r, "store", 0, k, v, [1, 2, 3, 1], seqs=[1, 1, 9, -1])             # twice, out of range
    both(c, r, "store", 0, k, v, [9, -1, 1, 0])                                # more than rows, negative, more than held
    assert flags_of(c) == r.flags == B.FLAG_BAD_SEQ | B.FLAG_BAD_LENGTH
    both(c, r, "fork", [0], [2])
    both(c, r, "store", 0, k, v, [3, 0, 3, 0])       # tokens 30..32: the first page is shared, the last is not
    assert flags_of(c) == r.flags == B.FLAG_BAD_SEQ | B.FLAG_BAD_LENGTH | B.FLAG_BAD_PAGE
    same_state(c, r)
    same_pool(c, r)


# ------------------------------------------------------------------ pages
def test_reserve_all_or_nothing_and_limits():
    c, r = pair(seqs=3, pages=6, max_pages=4)
    both(c, r, "reserve", [64, 33, 1])
    same_state(c, r)
    both(c, r, "reserve", [32, 0, 0])
    same_state(c, r)
    assert flags_of(c) == 0
    both(c, r, "reserve", [1, 40, 0])                   # two pages wanted, none free: nothing changes
    same_state(c, r)
    assert flags_of(c) == r.flags == B.FLAG_NO_PAGES
    both(c, r, "free", [1])
    both(c, r, "reserve", [33, 5, -1])                  # past max_pages; fits; negative
    same_state(c, r)
    assert flags_of(c) == r.flags == B.FLAG_NO_PAGES | B.FLAG_OVERFLOW | B.FLAG_BAD_LENGTH
    both(c, r, "reserve", [3, 4, 5], seqs=[2, 2, 7])
    same_state(c, r)
    assert flags_of(c) & B.FLAG_BAD_SEQ
    c.free(ints([0, 1, 1, 2])[:3])
    r.free([0, 1])
    same_state(c, r)
    with pytest.raises(DropKVError) as e:
        c.check()
    assert e.value.code == 7


@pytest.mark.parametrize("code,page,d,layers", [("e4m3", 32, 64, 2), ("int8", 64, 40, 1), ("int8", 32, 96, 2),
                                                ("e4m3", 128, 8, 1)])
@pytest.mark.parametrize("seed", [0, 1])
def test_random_program_matches_reference(code, page, d, layers, seed):
    """Random reserves, stores, forks, copies, compactions and frees, some of
    them impossible: state, codes and scales equal the reference after each."""
    rng = np.random.default_rng(seed)
    H, S = 2, 7
    c, r = pair(seqs=S, Hkv=H, d=d, pages=40, page=page, max_pages=5, layers=layers, code=code, seed=seed)
    for step in range(40):
        what = rng.choice(["grow", "grow", "fork", "copy", "compact", "free"])
        n = int(rng.integers(1, S + 1))
        some = [int(x) for x in rng.permutation(S)[:n]]
        if what == "grow":
            new = [int(rng.choice([0, 1, 2, page, page + 5])) for _ in some]
            before = list(r.length)
            both(c, r, "reserve", new, seqs=some)
            new = [r.length[s] - before[s] for s in some]
            if max(new) > 0:
                for layer in range(layers):
                    k, v = (draw_rows(n, H, max(new), d, 1000 * step + 2 * layer + j) for j in range(2))
                    both(c, r, "store", layer, k, v, new, seqs=some)
        elif what in ("fork", "copy"):
            src = [int(rng.integers(0, S)) for _ in range(n)]
            dst = [int(rng.integers(-1, S)) for _ in range(n)]
            both(c, r, what, src, dst)
        elif what == "compact":
            kept = [int(rng.integers(0, r.length[s] + 2)) if rng.random() < 0.9 else r.length[s] for s in some]
            stride = max(1, max(kept))
            idx = np.zeros((layers, n, H, stride), dtype=np.int64)
            for i, s in enumerate(some):
                for layer in range(layers):
                    for h in range(H):
                        m = min(kept[i], r.length[s])
                        pick = rng.permutation(r.length[s])[:m]
                        idx[layer, i, h, :m] = np.sort(pick) if rng.random() < 0.8 else pick
            c.compact(ints(idx.tolist()), ints(kept), ints(some))
            r.compact(idx.tolist(), kept, some)
        else:
            c.free(ints(some))
            r.free(some)
        same_state(c, r)
    same_pool(c, r)
    assert flags_of(c) == r.flags
    c.free(ints(list(range(S))))
    assert int(c.refs.abs().sum()) == 0


def test_fork_refusals_and_no_pages():
    c, r = pair(seqs=6, pages=9)
    fill(c, r, [70, 40, 0, 0, 0, 0])
    both(c, r, "fork", [0, 0, 1, 9, 2], [2, 2, 0, 3, 9])    # twice; a source as destination; out of range
    same_state(c, r)
    assert flags_of(c) == r.flags == B.FLAG_BAD_SEQ
    both(c, r, "copy", [0, 0], [3, 4])                      # six pages wanted, four free
    same_state(c, r)
    assert flags_of(c) == r.flags == B.FLAG_BAD_SEQ | B.FLAG_NO_PAGES
    both(c, r, "fork", [0], [1])                            # holds tokens
    both(c, r, "copy", [0], [3])
    same_state(c, r)
    same_pool(c, r)


def test_compact_refusals():
    c, r = pair(seqs=3, pages=12)
    fill(c, r, [70, 40, 10])
    before = c.k.clone()
    idx = torch.zeros(1, 3, 2, 80, dtype=torch.int32, device=DEV)
    c.compact(idx, ints([71, 41, -1]))                      # more than held, negative
    same_state(c, r)
    assert flags_of(c) == B.FLAG_BAD_K and torch.equal(before.view(torch.uint8), c.k.view(torch.uint8))
    c.reset_status()
    idx[0, 2, 1, 3] = 10                                    # a position outside the sequence: flagged, stored as zeros
    c.compact(idx[:, 2:], ints([5]), ints([2]))
    assert flags_of(c) == B.FLAG_BAD_K
    pg = c.table[2, 0].item()
    assert torch.all(c.k[0, pg, 1, 3].float() == 0) and c.length.tolist() == [70, 40, 5]


def test_damaged_tables_are_flagged():
    """Entries that are no pages, and counts that do not fit, are reported and never followed."""
    c, r = pair(seqs=3, pages=12, Hq=2)
    fill(c, r, [70, 40, 10])
    q = draw_rows(3, 2, 1, 64, 5).to(DEV)
    out = torch.full_like(q, 7.0)
    c.table[0, 1] = 12
    c.table[1, 0] = -3
    c.attention(0, q, out)
    assert flags_of(c) == B.FLAG_BAD_PAGE and torch.isfinite(out.float()).all()
    ref, vmax = r.attention(0, q.cpu().float().numpy())
    assert np.all(np.abs(out[2].cpu().double().numpy() - ref[2]) <= 0.02 * vmax[2][..., None])   # the others are served
    c.reset_status()
    c.store(0, q, q, ints([1, 1, 1]))
    assert flags_of(c) == 0                                  # their last pages are sound
    c.length[2] = 999
    c.attention(0, q, out)
    assert flags_of(c) & B.FLAG_BAD_LENGTH and torch.all(out[2] == 0)
    c.reset_status()
    c.free(ints([0, 1]))
    assert flags_of(c) == B.FLAG_BAD_PAGE
    c.reset_status()
    c.attention(0, q, out, seqs=ints([0, 5, -1]))
    assert flags_of(c) == B.FLAG_BAD_SEQ and torch.all(out == 0)


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("Hq,Hkv,d,page,T", [
    (4, 2, 64, 32, 1), (8, 1, 128, 64, 1), (7, 1, 96, 32, 2), (2, 2, 40, 32, 5), (32, 2, 16, 64, 1), (6, 3, 72, 128, 3),
    (3, 1, 8, 32, 9), (4, 4, 128, 128, 1), (5, 1, 112, 64, 8)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (37, 3), (64, 70), (500, 4)])
@pytest.mark.parametrize("room", [1, 8])
def test_attention_matches_reference(code, Hq, Hkv, d, page, T, window, sinks, room):
    """Sequences of 0, 1, a few and a few hundred tokens in one call; rows that
    see nothing; random bytes (not-a-number codes among them) in every slot
    that holds no token.  room: how many times longer the sequences could be
    (short units go to a CTA each, others are cut over the GPU)."""
    lengths = [0, 1, 3, page, page + 1, 211, 300]
    M = -(-300 // page)
    c, r = pair(seqs=7, Hkv=Hkv, d=d, pages=7 * M, page=page, max_pages=room * M, code=code, Hq=Hq, T=T, seed=d + T)
    fill(c, r, lengths, seed=T)
    q = draw_rows(7, Hq, T, d, 77, spread=0.3)
    check_attention(c, r, q, window=window, sinks=sinks)
    assert c.check() == 0


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("Hq,Hkv,d,page,T", [(7, 1, 96, 32, 2), (32, 2, 16, 64, 1), (3, 1, 8, 32, 9), (5, 1, 112, 64, 8),
                                             (9, 1, 128, 128, 1), (12, 1, 64, 32, 5)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (37, 3)])
def test_attention_with_room_for_long_sequences(code, Hq, Hkv, d, page, T, window, sinks):
    """The same lengths in a cache whose sequences could be hundreds of times
    longer: warps hold 16 rows."""
    test_attention_matches_reference(code, Hq, Hkv, d, page, T, window, sinks, 800)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_attention_long_split_over_the_gpu(code):
    """Lengths that are cut into many pieces, and a ragged batch of them."""
    c, r = pair(seqs=3, Hkv=2, d=128, pages=220, page=64, max_pages=160, code=code, Hq=8, T=2, seed=1)
    fill(c, r, [10000, 1, 3333], spread=0.2)
    q = draw_rows(3, 8, 2, 128, 4, spread=0.2)
    check_attention(c, r, q)
    check_attention(c, r, q, window=1000, sinks=5)
    check_attention(c, r, q[:2], seqs=[2, 0])
    check_attention(c, r, q[:2], seqs=[0, 0])
    check_attention(c, r, q[:1, :, :1].contiguous(), seqs=[2])


@pytest.mark.parametrize("Hq,Hkv,T,lengths", [(16, 2, 8, [2000, 5, 0, 700]), (24, 1, 7, [900, 901, 1, 64]),
                                              (40, 1, 40, [33, 500, 1500, 39]), (64, 1, 330, [400, 7, 0, 0])])
@pytest.mark.parametrize("room", [1, 8])
def test_attention_many_rows_per_head(Hq, Hkv, T, lengths, room):
    """Row groups: 56 to 21120 query rows of a KV head, more than a wave of warps."""
    M = -(-max(lengths) // 64)
    c, r = pair(seqs=4, Hkv=Hkv, d=64, pages=4 * M, page=64, max_pages=room * M, Hq=Hq, T=T, seed=T)
    fill(c, r, lengths, spread=0.3)
    q = draw_rows(4, Hq, T, 64, 5, spread=0.2)
    check_attention(c, r, q)
    check_attention(c, r, q, window=100, sinks=3)
    assert c.check() == 0


def test_attention_runs_of_many_tiles():
    """One sequence named 64 times: every warp walks over a hundred tiles and
    crosses sequences; all copies get the reference's output, and the same bytes
    whatever their place in the call but for where runs cut them."""
    c, r = pair(seqs=64, Hkv=4, d=128, pages=170, page=128, max_pages=170, Hq=8, T=1, seed=2)
    fill(c, r, [20001], spread=0.2)
    q = draw_rows(1, 8, 1, 128, 4, spread=0.2)
    one = check_attention(c, r, q, seqs=[0])
    out = torch.zeros(64, 8, 1, 128, dtype=torch.bfloat16, device=DEV)
    c.attention(0, q.to(DEV).expand(64, -1, -1, -1).contiguous(), out, seqs=ints([0] * 64))
    # two orders of summation differ by at most a bf16 step and the bound's fp16 terms
    far = (out.float() - one.float()).abs()
    top = float(np.abs(r.values(0, 0, 0)[1]).max())
    assert float(far.max()) <= 2.0 ** -7 * float(one.float().abs().max()) + 2.0 ** -9 * top
    assert c.check() == 0


def test_offsets_past_32_bits():
    """A pool of 5 GiB of K codes: the same calls on pages behind the 4 GiB line
    and on the first pages give the same bytes."""
    P, page, H, d = 41000, 128, 8, 128
    big = PagedCache(4, H, d, P, page, 8, Hq=16, T=1, device=DEV)
    small = PagedCache(4, H, d, 40, page, 8, Hq=16, T=1, device=DEV)
    big.refs[:P - 40] = 1                                  # the last 40 pages are free
    rows = [draw_rows(2, H, 300, d, 5 + i).to(DEV) for i in range(2)]
    q = draw_rows(3, 16, 1, d, 9).to(DEV)
    idx = ints(np.sort(np.stack([np.random.default_rng(h).permutation(300)[:200] for h in range(H)]), -1)[None, None].tolist())
    outs = []
    for c in (big, small):
        c.reserve(ints([300, 40]))
        c.store(0, rows[0], rows[1], ints([300, 40]))
        c.fork(ints([0]), ints([2]))
        c.copy(ints([1]), ints([3]))
        c.compact(idx, ints([200]), ints([2]))
        out = torch.zeros_like(q)
        c.attention(0, q, out, seqs=ints([0, 2, 3]))
        assert c.check() == 0
        outs.append(out)
    assert torch.equal(outs[0], outs[1])
    assert torch.equal(torch.where(small.table >= 0, small.table + P - 40, small.table), big.table)
    assert torch.equal(big.refs[P - 40:], small.refs)
    for a, b in ((big.k, small.k), (big.v, small.v)):
        assert torch.equal(a[:, P - 40:].view(torch.uint8), b.view(torch.uint8))


def test_attention_many_sequences():
    n = 150
    lengths = [(i * 37) % 130 for i in range(n)]
    c, r = pair(seqs=n, Hkv=1, d=32, pages=n * 5, page=32, max_pages=5, Hq=3, T=1)
    fill(c, r, lengths)
    q = draw_rows(n, 3, 1, 32, 8)
    check_attention(c, r, q)
    check_attention(c, r, q, seqs=[(i * 7) % n for i in range(n)])


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("Hq,Hkv,d,T,n", [(8, 4, 64, 1, 90), (12, 2, 128, 3, 100), (16, 8, 64, 8, 90), (33, 3, 72, 2, 120),
                                          (9, 1, 16, 5, 330)])
def test_attention_many_short_sequences(code, Hq, Hkv, d, T, n):
    """A warp per unit and row group (8 or 16 rows): empty sequences, fewer
    tokens than rows, numbers that are no sequence, and with room for long ones
    where a window bounds what is read."""
    lengths = [(i * 37) % 150 if i % 9 else 0 for i in range(n)]
    q = draw_rows(n, Hq, T, d, 8, spread=0.3)
    for room, masks in ((5, ((0, 0), (1, 0), (40, 5), (64, 100))), (400, ((1, 0), (40, 5), (64, 100)))):
        c, r = pair(seqs=n, Hkv=Hkv, d=d, pages=n * 5, page=32, max_pages=room, code=code, Hq=Hq, T=T)
        fill(c, r, lengths, spread=0.3)
        for window, sinks in masks:
            check_attention(c, r, q, window=window, sinks=sinks)
        order = [(i * 7 + 3) % n for i in range(n)]
        out = check_attention(c, r, q, window=40, sinks=5, seqs=order)
        assert c.check() == 0
        order[4], order[n - 1] = n, -1
        got = torch.full_like(out, 7.0)
        c.attention(0, q.to(DEV), got, window=40, sinks=5, seqs=ints(order))
        assert flags_of(c) == B.FLAG_BAD_SEQ
        for i in range(n):
            assert torch.equal(got[i], out[i]) if i not in (4, n - 1) else torch.all(got[i] == 0)


def test_attention_scales_and_logits_of_very_different_size():
    """Value pages 2^40 apart, one key far above the rest, constant and zero rows."""
    c, r = pair(seqs=2, Hkv=1, d=64, pages=24, page=32, max_pages=12, Hq=2, T=1)
    both(c, r, "reserve", [300, 310])
    k, v = draw_rows(2, 1, 310, 64, 1), draw_rows(2, 1, 310, 64, 2)
    v[:, :, 64:96] *= 2.0 ** 20
    v[:, :, 96:128] *= 2.0 ** -20
    v[:, :, 160:192] = 0.0
    k[1, 0, 100] *= 6.0
    k[0, 0, 200:] = 0.0
    both(c, r, "store", 0, k, v, [300, 310])
    q = draw_rows(2, 2, 1, 64, 3)
    q[0, 1] = 0.0
    q[1, 1] = k[1, 0, 100] * 0.5
    check_attention(c, r, q)


def test_not_a_number_reaches_only_its_head():
    c, r = pair(seqs=2, Hkv=2, d=64, pages=24, max_pages=12, Hq=2, T=1)
    both(c, r, "reserve", [100, 90])
    k, v = draw_rows(2, 2, 100, 64, 1), draw_rows(2, 2, 100, 64, 2)
    v[0, 1, 50, 3] = float("nan")
    both(c, r, "store", 0, k, v, [100, 90])
    q = draw_rows(2, 2, 1, 64, 3).to(DEV)
    out = torch.zeros_like(q)
    c.attention(0, q, out)
    bad = torch.isnan(out.float()).any(-1)[..., 0].cpu()
    assert bad.tolist() == [[False, True], [False, False]]
    c.attention(0, q, out, window=49)                        # token 50 is out of the window of 49 ending at 99
    assert torch.isfinite(out.float()).all()


# ------------------------------------------------------------------ how it is called
def test_refusals_of_arguments():
    c = PagedCache(3, 2, 64, 12, 32, 4, Hq=4, T=2, device=DEV)
    q = torch.zeros(3, 4, 2, 64, dtype=torch.bfloat16, device=DEV)
    out = torch.zeros_like(q)
    bad = [lambda: c.attention(1, q, out), lambda: c.attention(0, q.float(), out.float()),
           lambda: c.attention(0, q.cpu(), out), lambda: c.attention(0, q[:, :2].contiguous(), out[:, :2].contiguous()),
           lambda: c.attention(0, torch.cat((q, q), 2), torch.cat((q, q), 2)),
           lambda: c.attention(0, q.transpose(1, 2).contiguous().transpose(1, 2), out),
           lambda: c.attention(0, torch.cat((q, q)), torch.cat((q, q))), lambda: c.attention(0, q, out[:2]),
           lambda: c.reserve(torch.zeros(4, dtype=torch.int32, device=DEV)),
           lambda: c.reserve(torch.zeros(3, dtype=torch.int64, device=DEV)),
           lambda: c.store(0, q[:, :1], q[:, :1]), lambda: c.fork(ints([0, 1]), ints([2])),
           lambda: c.compact(torch.zeros(1, 3, 1, 8, dtype=torch.int32, device=DEV), ints([1, 1, 1])),
           lambda: c.free(ints([0, 1, 2, 0])), lambda: PagedCache(3, 2, 64, 12, code="e5m2", device=DEV)]
    for call in bad:
        with pytest.raises((ValueError, KeyError)):
            call()
    for kw in (dict(window=-1), dict(sinks=-1)):
        with pytest.raises(DropKVError) as e:
            c.attention(0, q, out, **kw)
        assert e.value.code == 1
    with pytest.raises(DropKVError) as e:                    # in place: the output is read again by other rows
        c.attention(0, q, q)
    assert e.value.code == 1
    for kw in (dict(d=60), dict(d=136), dict(page=48), dict(pages=0), dict(Hq=3)):
        with pytest.raises(DropKVError) as e:
            PagedCache(**{**dict(seqs=3, Hkv=2, d=64, pages=12, device=DEV), **kw})
        assert e.value.code == 6
    with pytest.raises(ValueError):
        c.attention(0, q, out, window=1 << 32)
    with pytest.raises(ValueError):
        c.attention(0, q, out, window=-(1 << 32) + 5)
    c.attention(0, q[:0], out[:0])
    torch.cuda.synchronize()
    assert flags_of(c) == 0 and torch.all(out == 0)


def test_calls_with_nothing_to_do():
    """No entries, no rows, nothing kept: empty tensors have no address."""
    c, r = pair(seqs=3, max_pages=4, Hq=2)
    both(c, r, "reserve", [40, 0, 64])
    k = draw_rows(3, 2, 64, 64, 1)
    both(c, r, "store", 0, k, k, [40, 0, 64])
    none = ints([])
    c.reserve(none, seqs=none)
    c.store(0, k[:0].to(DEV), k[:0].to(DEV))
    c.store(0, k[:, :, :0].to(DEV), k[:, :, :0].to(DEV))
    c.fork(none, none)
    c.copy(none, none)
    c.compact(torch.zeros(1, 0, 2, 4, dtype=torch.int32, device=DEV), none)
    c.free(none)
    same_state(c, r)
    same_pool(c, r)
    c.compact(torch.zeros(1, 2, 2, 0, dtype=torch.int32, device=DEV), ints([0, 0]), seqs=ints([0, 1]))   # keeps nothing
    assert c.length.tolist() == [0, 0, 64] and c.count.tolist() == [0, 0, 2] and sum(c.refs.tolist()) == 2
    c.compact(torch.zeros(1, 1, 2, 0, dtype=torch.int32, device=DEV), ints([1]), seqs=ints([2]))          # keeps more
    assert flags_of(c) == B.FLAG_BAD_K and c.length.tolist() == [0, 0, 64]


def test_streams_graphs_and_repeats_give_the_same_bytes():
    c, r = pair(seqs=4, Hkv=2, d=128, pages=120, page=64, max_pages=40, Hq=8, T=1)
    fill(c, r, [2500, 17, 640, 1300])
    q = draw_rows(4, 8, 1, 128, 5).to(DEV)
    want = torch.zeros_like(q)
    c.attention(0, q, want)
    for _ in range(5):
        out = torch.zeros_like(q)
        c.attention(0, q, out)
        assert torch.equal(out, want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(q)
    with torch.cuda.stream(st):
        c.attention(0, q, out)
    c.attention(0, q, out, stream=st)
    st.synchronize()
    assert torch.equal(out, want)
    # a captured step (reserve, store, attention, fork, free), replayed twice, equals eager steps
    rows = [draw_rows(4, 2, 1, 128, 60 + j).to(DEV) for j in range(2)]
    one, src, dst = ints([1, 0, 1, 1]), ints([0]), ints([1])
    eager = PagedCache(4, 2, 128, 120, 64, 40, Hq=8, device=DEV)
    for name in ("k", "v", "k_scale", "v_scale", "refs", "table", "count", "length"):
        getattr(eager, name).copy_(getattr(c, name))

    def step(cache, res):
        cache.free(dst)
        cache.fork(src, dst)
        cache.reserve(one)
        cache.store(0, rows[0], rows[1], one)
        cache.attention(0, q, res)

    a, b = torch.zeros_like(q), torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c, a)
    for _ in range(2):
        graph.replay()
        step(eager, b)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    for name in ("k", "v", "k_scale", "v_scale", "refs", "table", "count", "length"):
        assert torch.equal(getattr(c, name).view(torch.uint8), getattr(eager, name).view(torch.uint8)), name


def test_two_caches_on_two_streams():
    made = [pair(seqs=2, Hkv=2, d=128, pages=100, page=64, max_pages=50, Hq=4, T=1, seed=s, code=code)
            for s, code in ((1, "e4m3"), (2, "int8"))]
    for c, r in made:
        fill(c, r, [3000, 777])
    q = draw_rows(2, 4, 1, 128, 5)
    torch.cuda.synchronize()
    outs, streams = [], [torch.cuda.Stream() for _ in made]
    qd = q.to(DEV)
    torch.cuda.synchronize()
    for (c, _), st in zip(made, streams):
        out = torch.zeros_like(qd)
        torch.cuda.synchronize()
        outs.append(out)
    for _ in range(20):
        for (c, _), st, out in zip(made, streams, outs):
            c.attention(0, qd, out, stream=st)
    torch.cuda.synchronize()
    for (c, r), out in zip(made, outs):
        again = torch.zeros_like(qd)
        c.attention(0, qd, again)
        assert torch.equal(again, out)
        check_attention(c, r, q)
