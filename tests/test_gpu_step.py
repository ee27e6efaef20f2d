"""Norms and positions, the store that applies them and the reading back, on
the GPU: against the formulas in 64 bits, and the one call against the two.

Bound of a rotated channel, with y the normed values of its pair in 64 bits and
A the amplitude: the result is rounded to bf16 (2^-8 of itself); cosine and
sine are off by 2^-19 each, so the channel by 2^-19 A (|y_a| + |y_b|); the norm
and the products are fp32, a sum of at most 16 + 4 terms in order under a square
root and five products: below 2^-19 of either y.  Together 2^-8 |o| + 2^-18 A
(|y_a| + |y_b|), and a margin of 1/64 for the rounding of these errors themselves."""
import numpy as np
import pytest
import torch

from kv_cache_eviction_dropkv_gb300 import DropKVError, Rotary, _binding as B
from tests.test_gpu_paged import DEV, draw_rows, fill, flags_of, ints, pair
from tests.test_step_boundary import by_formula

gpu = pytest.mark.gpu
pytestmark = gpu
EPS = 1e-6


def rows(n, heads, length, d, seed, packed=False):
    """bf16 rows [n][heads][length][d] on the device; packed: a view of token-major ones."""
    x = draw_rows(n, length if packed else heads, heads if packed else length, d, seed).to(DEV)
    return x.transpose(1, 2) if packed else x


def weights(d, seed):
    return 1.0 + 0.25 * torch.randn(d, generator=torch.Generator().manual_seed(seed))


def reference(x, weight, positions, d, dims, layout, base, kind, kw):
    """Rotated rows in 64 bits and the bound; x [n][heads][rows][d], positions [n][rows]."""
    y = x.detach().cpu().double().numpy()
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + EPS) * weight.double().numpy()
    o, size = y.copy(), np.zeros_like(y)
    amplitude = 1.0
    if dims:
        f, amplitude = by_formula(dims, base, kind, **kw)
        # whole turns leave before the angle is rounded: far positions stay exact
        turn = np.mod(np.asarray(positions, dtype=np.longdouble)[..., None] * np.asarray(f, dtype=np.longdouble)
                      / (2 * np.longdouble(np.pi)), 1.0).astype(np.float64) * 2 * np.pi
        c, s = (amplitude * g(turn)[:, None] for g in (np.cos, np.sin))
        at = (slice(0, dims // 2), slice(dims // 2, dims)) if layout == "half" else (slice(0, dims, 2), slice(1, dims, 2))
        a, b = y[..., at[0]], y[..., at[1]]
        o[..., at[0]], o[..., at[1]] = a * c - b * s, b * c + a * s
        size[..., at[0]] = size[..., at[1]] = amplitude * (np.abs(a) + np.abs(b))
    size[..., dims:] = np.abs(y[..., dims:])
    return o, (1 + 1 / 64) * (2.0 ** -8 * np.abs(o) + 2.0 ** -18 * size) + 2.0 ** -133


def near(got, want, bound, lengths=None, kept=None):
    got = got.cpu().double().numpy()
    for b in range(len(got)):
        n = got.shape[2] if lengths is None else lengths[b]
        err = np.abs(got[b, :, :n] - want[b, :, :n])
        assert np.all(err <= bound[b, :, :n]), float((err / bound[b, :, :n]).max())
        if kept is not None:
            assert np.all(got[b, :, n:] == kept)


CASES = [
    # B Hq Hkv n   d  dims  layout         norms  scaling                                      packed
    (1, 4, 2, 1, 64, 64, "half", True, None, {}, False),
    (3, 5, 1, 7, 128, 128, "half", True, "bands", dict(factor=8.0, original=8192), True),
    (2, 8, 8, 33, 96, 48, "interleaved", False, "yarn", dict(factor=16.0, original=4096), True),
    (1, 1, 1, 130, 8, 8, "half", True, "linear", dict(factor=4.0), False),
    (2, 3, 3, 17, 40, 40, "half", False, None, {}, True),
    (2, 12, 4, 19, 72, 24, "half", True, "ntk", dict(factor=8.0), False),
    (1, 32, 8, 65, 128, 64, "interleaved", True, None, {}, True),
    (70, 9, 3, 1, 80, 32, "half", True, None, {}, True),
    (4, 2, 2, 5, 112, 0, "half", True, None, {}, False),
    (1, 40, 8, 300, 16, 16, "interleaved", True, None, {}, True),
    (5, 33, 11, 3, 120, 104, "half", False, None, {}, False),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("where", ["none", "first", "each"])
def test_rotation(case, where):
    n_seq, Hq, Hkv, n, d, dims, layout, norms, kind, kw, packed = case
    q, k = rows(n_seq, Hq, n, d, 1, packed), rows(n_seq, Hkv, n, d, 2, packed)
    qw, kw_ = (weights(d, 3), weights(d, 4)) if norms else (None, None)
    base = 500000.0
    plan = Rotary(d, dims=dims, base=base, layout=layout, scaling=dict(kind=kind, **kw) if kind else None,
                  q_norm=qw, k_norm=kw_, eps=EPS, device=DEV)
    rng = np.random.default_rng(5)
    t = np.arange(n)
    if where == "none":
        positions, at = None, np.tile(t, (n_seq, 1))
    elif where == "first":
        first = rng.integers(-3, 200000, n_seq)
        first[-1] = 2 ** 31 - 1 - n
        positions, at = ints(first.tolist()), first[:, None] + t
    else:
        at = rng.integers(-2 ** 31, 2 ** 31, (n_seq, n))
        positions = ints(at.tolist())
    lengths = [(n * (b + 1)) // n_seq if b else 0 for b in range(n_seq)] if n_seq > 1 else [n]
    q_out, k_out = torch.full((n_seq, Hq, n, d), 7.0, dtype=torch.bfloat16, device=DEV), \
        torch.full((n_seq, Hkv, n, d), 7.0, dtype=torch.bfloat16, device=DEV)
    plan.apply(q, k, q_out, k_out, positions=positions, lengths=ints(lengths))
    assert plan.check() == 0
    for x, w, out in ((q, qw, q_out), (k, kw_, k_out)):
        near(out, *reference(x, w, at, d, dims, layout, base, kind, kw), lengths, 7.0)


def test_rotation_in_place_alone_and_broadcast():
    plan = Rotary(64, q_norm=weights(64, 1), k_norm=weights(64, 2), device=DEV)
    q, k = rows(2, 6, 9, 64, 1), rows(2, 2, 9, 64, 2)
    q_out, k_out = torch.empty_like(q), torch.empty_like(k)
    plan.apply(q, k, q_out, k_out)
    q2, k2 = q.clone(), k.clone()
    plan.apply(q2, None, q2, None)
    plan.apply(None, k2, None, k2)
    assert torch.equal(q2, q_out) and torch.equal(k2, k_out)
    # one row for all heads, without a copy
    one = q[:, :1].expand(2, 6, 9, 64)
    a, b = torch.empty_like(q), torch.empty_like(q)
    plan.apply(one, None, a, None)
    plan.apply(one.contiguous(), None, b, None)
    assert torch.equal(a, b)
    # views with gaps: every other token of a longer batch, heads of a packed projection
    wide = torch.randn(2, 18, 10, 64, device=DEV).bfloat16()
    view = wide[:, ::2, 2:8].transpose(1, 2)
    plan.apply(view, None, a, None)
    plan.apply(view.contiguous(), None, b, None)
    assert torch.equal(a, b)
    # nothing to do
    plan.apply(q[:0], None, q_out[:0], None)
    plan.apply(q[:, :, :0], None, q_out[:, :, :0], None)
    plan.apply(None, None, None, None)
    assert plan.check() == 0


def test_rotation_of_extreme_rows():
    """Squares past fp32, rows of zeros, infinities and not-a-number: each row is its own."""
    d = 128
    w = weights(d, 1)
    plan = Rotary(d, q_norm=w, device=DEV)
    x = draw_rows(1, 1, 8, d, 3)
    x[0, 0, 1] *= 2.0 ** 100                              # the sum of squares passes fp32
    x[0, 0, 2] = 0.0
    x[0, 0, 3] *= 2.0 ** -100                             # eps rules
    x[0, 0, 4, 5] = float("inf")
    x[0, 0, 5, 6] = float("nan")
    x[0, 0, 6] = 3.0e38
    out = torch.empty(1, 1, 8, d, dtype=torch.bfloat16, device=DEV)
    plan.apply(x.to(DEV), None, out, None)
    got = out.cpu().double().numpy()[0, 0]
    fine = [0, 1, 2, 3, 6, 7]
    want, bound = reference(x[:, :, fine], w, np.array([fine]), d, d, "half", 10000.0, None, {})
    assert np.all(np.abs(got[fine] - want[0, 0]) <= bound[0, 0])
    assert np.isnan(got[4]).any() and np.isnan(got[5]).all()
    assert plan.check() == 0


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_channels_that_do_not_turn_keep_to_themselves(layout):
    x = draw_rows(1, 2, 3, 64, 3)
    x[..., 40], x[..., 63] = float("inf"), float("nan")
    out = torch.empty(1, 2, 3, 64, dtype=torch.bfloat16, device=DEV)
    for dims in (0, 16, 32):
        Rotary(64, dims=dims, layout=layout, device=DEV).apply(x.to(DEV), None, out, None, positions=ints([1000]))
        # (a not-a-number leaves the rounding as the canonical one)
        torch.testing.assert_close(out[..., 32:].cpu(), x[..., 32:], rtol=0, atol=0, equal_nan=True)
        assert bool(out[..., :32].isfinite().all())


def test_rotation_refusals():
    plan = Rotary(64, device=DEV)
    q, k = rows(2, 4, 3, 64, 1), rows(2, 2, 3, 64, 2)
    q_out, k_out = torch.zeros_like(q), torch.zeros_like(k)
    for bad in (dict(q=q.float()), dict(q=q[..., :32]), dict(q=q.cpu()), dict(q_out=q_out[:, :2]), dict(k=k[:1]),
                dict(q_out=torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16, device=DEV).transpose(1, 2)),
                dict(positions=ints([1])), dict(positions=ints([[1, 2], [3, 4]])), dict(lengths=ints([3])),
                dict(positions=torch.zeros(2, dtype=torch.int64, device=DEV))):
        with pytest.raises(ValueError):
            plan.apply(**{**dict(q=q, k=k, q_out=q_out, k_out=k_out), **bad})
    packed = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(DropKVError):                      # an output over an input of another order
        plan.apply(packed.transpose(1, 2), None, packed.view(2, 4, 3, 64), None)
    assert torch.equal(q_out, torch.zeros_like(q)) and plan.check() == 0
    plan.apply(q, k, q_out, k_out, lengths=ints([4, -1]))
    assert torch.equal(q_out, torch.zeros_like(q))
    assert int(plan.status.item()) == B.FLAG_BAD_LENGTH
    plan.reset_status()
    plan.apply(q, k, q_out, k_out, lengths=ints([-5, 2]))  # the other sequence is served
    want = torch.zeros_like(q)
    fresh = Rotary(64, device=DEV)
    fresh.apply(q[1:], None, want[1:], None, lengths=ints([2]))
    assert torch.equal(q_out, want) and int(plan.status.item()) == B.FLAG_BAD_LENGTH


# ------------------------------------------------------------------ store with rotation
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("page,d,Hkv,g,dims,layout", [
    (32, 8, 3, 2, 8, "half"), (32, 96, 1, 7, 48, "interleaved"), (64, 40, 2, 1, 24, "half"), (64, 128, 2, 4, 128, "half"),
    (128, 72, 1, 3, 72, "half"), (128, 128, 2, 2, 64, "interleaved"), (64, 64, 1, 2, 0, "half")])
def test_store_rotated_is_rotation_and_store(code, page, d, Hkv, g, dims, layout):
    """Prompts of no, one and many tokens, then single ones and runs behind
    partly filled pages: the same bytes, and the same queries, as in two calls."""
    one, _ = pair(seqs=5, Hkv=Hkv, d=d, pages=30, page=page, max_pages=6, layers=2, code=code, seed=d)
    two, _ = pair(seqs=5, Hkv=Hkv, d=d, pages=30, page=page, max_pages=6, layers=2, code=code, seed=d)
    plan = Rotary(d, dims=dims, layout=layout, q_norm=weights(d, 1) if page != 64 else None, k_norm=weights(d, 2),
                  device=DEV)
    for step in range(5):
        new = [[0, 1, page - 1, page, 2 * page + 3], [1, 1, 1, 1, 1], [3, 0, 2, page, 1], [1, 2, 0, 1, 40],
               [1, 1, 1, 1, 1]][step]
        for c in (one, two):
            c.reserve(ints(new))
        length = max(new)
        q, k, v = (rows(5, h, length, d, 10 * step + j, packed=step % 2 == 0)
                   for j, h in enumerate((g * Hkv, Hkv, Hkv)))
        k = k * 2.0 ** (step - 1)                          # louder and louder: most scales grow
        start = one.length - ints(new)
        at = [None, ints([7, 100000, 0, 5, -9]), (start[:, None] + torch.arange(length, device=DEV)).to(torch.int32),
              None, None][step]
        q_out = torch.full((5, g * Hkv, length, d), 7.0, dtype=torch.bfloat16, device=DEV)
        q_two, k_two = q_out.clone(), torch.zeros(5, Hkv, length, d, dtype=torch.bfloat16, device=DEV)
        one.store_rotated(step % 2, plan, q, k, v, q_out, positions=at, counts=ints(new))
        plan.apply(q, k, q_two, k_two, positions=start if at is None else at, lengths=ints(new))
        two.store(step % 2, k_two, v.contiguous(), ints(new))
        assert torch.equal(q_out, q_two)
        for a, b in ((one.k, two.k), (one.v, two.v)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert torch.equal(one.k_scale, two.k_scale) and torch.equal(one.v_scale, two.v_scale)
    assert one.check() == two.check() == plan.check() == 0


def test_store_rotated_flags_and_defaults():
    c, _ = pair(seqs=4, Hkv=2, d=64, page=32, seed=2)
    plan = Rotary(64, device=DEV)
    c.reserve(ints([5, 40, 0, 33]))
    q, k, v = rows(4, 4, 5, 64, 1), rows(4, 2, 5, 64, 2), rows(4, 2, 5, 64, 3)
    q_out = torch.full_like(q, 7.0)
    before = c.k.view(torch.uint8).clone()
    # a sequence named twice is served for its first entry, one that is not there for none, and so are their queries
    c.store_rotated(0, plan, q, k, v, q_out, counts=ints([5, 5, 5, 5]), seqs=ints([1, 1, 9, 2]))
    assert flags_of(c) == B.FLAG_BAD_SEQ | B.FLAG_BAD_LENGTH       # sequence 2 is empty
    assert torch.all(q_out[1:] == 7.0) and not torch.any(q_out[0] == 7.0)
    pages = c.table[1, :2].long()
    other = torch.ones(c.pages, dtype=torch.bool, device=DEV)
    other[pages] = False
    assert torch.equal(c.k.view(torch.uint8)[0, other], before[0, other])
    assert not torch.equal(c.k.view(torch.uint8)[0, pages], before[0, pages])
    c.reset_status()
    # without queries
    d2, _ = pair(seqs=4, Hkv=2, d=64, page=32, seed=2)
    d2.reserve(ints([5, 40, 0, 33]))
    d2.store_rotated(0, plan, None, k[:1], v[:1], None, counts=ints([5]), seqs=ints([1]))
    assert torch.equal(c.k.view(torch.uint8), d2.k.view(torch.uint8)) and torch.equal(c.v.view(torch.uint8), d2.v.view(torch.uint8))
    # a shared page is not written; infinities are flagged and take no part in the scale
    c.fork(ints([3]), ints([2]))
    c.store_rotated(0, plan, q[:1], k[:1], v[:1], q_out[:1], counts=ints([5]), seqs=ints([3]))
    assert flags_of(c) == B.FLAG_BAD_PAGE
    c.reset_status()
    v[0, 0, 1, 3] = float("inf")
    c.store_rotated(0, plan, q[:1], k[:1], v[:1], q_out[:1], counts=ints([2]), seqs=ints([0]))
    assert flags_of(c) == B.FLAG_NONFINITE
    c.reset_status()
    for bad in (dict(k=k.float()), dict(v=v[:, :1]), dict(q_out=q_out[..., :32]), dict(layer=1), dict(counts=ints([1])),
                dict(positions=ints([[1]])), dict(rotary=Rotary(128, device=DEV)), dict(q=q[:, :, :2])):
        with pytest.raises((ValueError, AttributeError)):
            c.store_rotated(**{**dict(layer=0, rotary=plan, q=q, k=k, v=v, q_out=q_out), **bad})
    with pytest.raises(DropKVError):
        c.store_rotated(0, plan, q, k, v, q)
    c.store_rotated(0, plan, q[:, :0], k, v, q_out[:, :0], counts=ints([0, 0, 0, 0]))
    assert c.check() == 0


# ------------------------------------------------------------------ reading back
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("page,d,Hkv", [(32, 8, 3), (32, 96, 1), (64, 40, 2), (64, 128, 2), (128, 72, 1), (128, 128, 1)])
def test_read_gives_code_times_scale(code, page, d, Hkv):
    c, r = pair(seqs=6, Hkv=Hkv, d=d, pages=40, page=page, max_pages=8, layers=2, code=code, seed=d)
    lengths = [0, 1, page - 1, page, 2 * page + 3, 7 * page + 5]
    fill(c, r, lengths, seed=1)
    seqs = [5, 4, 3, 2, 1, 0]
    for starts, counts in ((None, None), ([0] * 6, [3, 2, 1, 0, 1, 0]), ([page - 1, page + 1, 5, 0, 0, 0], None),
                           ([6 * page + 7, 2 * page + 2, page, 3, 1, 0], [page - 7, 1, 0, page - 5, 0, 0])):
        have = [lengths[s] for s in seqs]
        a = [0] * 6 if starts is None else starts
        want = [h - x for h, x in zip(have, a)] if counts is None else counts
        length = max(want) + 3
        k, v = (torch.full((6, Hkv, length, d), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        c.read(1, k, v, starts=None if starts is None else ints(starts), counts=None if counts is None else ints(counts),
               seqs=ints(seqs))
        assert c.check() == 0
        for i, s in enumerate(seqs):
            for h in range(Hkv):
                for out, x in zip((k, v), r.values(1, s, h)):
                    rounded = torch.from_numpy(x[a[i]:a[i] + want[i]]).float().bfloat16()
                    if code == "int8":        # the product is rounded to fp32 first
                        exact = torch.from_numpy(x[a[i]:a[i] + want[i]])
                        err = (out[i, h, :want[i]].cpu().double() - exact).abs()
                        assert bool((err <= exact.abs() * (2.0 ** -8 + 2.0 ** -23)).all())
                    else:
                        assert torch.equal(out[i, h, :want[i]].cpu(), rounded)
                    assert bool((out[i, h, want[i]:] == 7.0).all())


def test_read_flags_and_refusals():
    c, r = pair(seqs=4, Hkv=2, d=64, page=32, seed=4)
    fill(c, r, [5, 70, 0, 33])
    k, v = (torch.full((4, 2, 40, 64), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    none = k.clone()

    def flags(**kw):
        k.fill_(7.0), v.fill_(7.0)
        c.read(0, k, v, **kw)
        f = flags_of(c)
        c.reset_status()
        return f

    assert flags() == B.FLAG_BAD_LENGTH and torch.equal(k[1], none[1]) and not torch.equal(k[0], none[0])   # 70 > 40 rows
    assert flags(seqs=ints([-1, 4, 0, 0])) == B.FLAG_BAD_SEQ and torch.equal(k[:2], none[:2])
    assert torch.equal(k[2], k[3]) and not torch.equal(k[2], none[2])        # named twice: both are served
    for starts, counts in (([6, 71, 1, 34], None), ([-1, -1, -1, -1], [1, 1, 1, 1]), ([0, 0, 0, 0], [6, 41, 1, -1]),
                           ([5, 70, 0, 33], [1, 1, 1, 1]), ([2 ** 31 - 1] * 4, [2 ** 31 - 1] * 4)):
        got = flags(starts=ints(starts), counts=None if counts is None else ints(counts))
        assert got == B.FLAG_BAD_LENGTH and torch.equal(k, none) and torch.equal(v, none)
    assert flags(starts=ints([5, 70, 0, 33])) == 0 and torch.equal(k, none)                          # no tokens
    c.table[1, 1] = -1
    assert flags(starts=ints([0, 31, 0, 0]), counts=ints([0, 39, 0, 0])) == B.FLAG_BAD_PAGE
    assert torch.equal(k[1, :, 1:33], none[1, :, 1:33]) and not torch.equal(k[1, :, 0], none[1, :, 0])
    for bad in (dict(v_out=v[:, :1]), dict(k_out=k.float()), dict(starts=ints([1])), dict(layer=1), dict(seqs=ints([1]))):
        with pytest.raises(ValueError):
            c.read(**{**dict(layer=0, k_out=k, v_out=v), **bad})
    with pytest.raises(DropKVError):
        c.read(0, k, k)
    c.read(0, k[:, :, :0], v[:, :, :0]), c.read(0, k[:0], v[:0])
    assert c.check() == 0


def test_step_calls_on_streams_and_in_graphs():
    """Captured once, replayed on new inputs in the same buffers; on a stream of its own."""
    c, r = pair(seqs=3, Hkv=2, d=64, page=32, seed=6)
    other, _ = pair(seqs=3, Hkv=2, d=64, page=32, seed=6)
    plan = Rotary(64, q_norm=weights(64, 1), device=DEV)
    new = ints([4, 1, 0])
    for x in (c, other):
        x.reserve(ints([4, 33, 0]))
    q, k, v = rows(3, 4, 4, 64, 1), rows(3, 2, 4, 64, 2), rows(3, 2, 4, 64, 3)
    q_out, k_out, v_out = torch.zeros_like(q), torch.zeros(3, 2, 40, 64, dtype=torch.bfloat16, device=DEV), \
        torch.zeros(3, 2, 40, 64, dtype=torch.bfloat16, device=DEV)

    def step(cache, to, ko, vo, stream=None):
        cache.store_rotated(0, plan, q, k, v, to, counts=new, stream=stream)
        cache.read(0, ko, vo, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(c, q_out, k_out, v_out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c, q_out, k_out, v_out)
    for seed in (10, 20):
        for t, h in ((q, 4), (k, 2), (v, 2)):
            t.copy_(rows(3, h, 4, 64, seed + h))
        graph.replay()
        torch.cuda.synchronize()
        a, b, d2 = torch.zeros_like(q), torch.zeros_like(k_out), torch.zeros_like(v_out)
        step(other, a, b, d2, stream=side)
        side.synchronize()
        for got, want in ((a, q_out), (b, k_out), (d2, v_out)):     # (bits: slots never stored may hold not-a-number)
            assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    assert c.check() == 0 and other.check() == 0
