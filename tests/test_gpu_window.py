"""The windowed prompt attention against the plain reference in 64 bits.

Bound per element: the output is rounded to bf16 (2^-8 |o|), each probability
enters the product as bf16 (2^-8 of itself: at most 2^-8 V after the division
by the sum, V the largest |v| the row sees); 2^-6 of that covers the fp32
arguments and sums (below 2^-14 relative at these sizes)."""
import numpy as np
import pytest
import torch

from kv_cache_eviction_dropkv_gb300 import DropKV, DropKVError, _binding as B, _build
from tests import _paged as R

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0) if torch.cuda.is_available() else None


def _inputs(B_, Hq, Hkv, d, n, lengths, seed=0):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(B_, h, n, d, generator=g).bfloat16() for h in (Hq, Hkv, Hkv))
    for b, L in enumerate(lengths):
        q[b, :, L:] = float("nan")
        k[b, :, L:] = float("nan")
        v[b, :, L:] = float("inf")
    return q, k, v


def _check(op, q, k, v, lengths, window, sinks):
    out = torch.full(q.shape, -7.25, dtype=torch.bfloat16, device=DEV)
    op.window_attention(q.to(DEV), k.to(DEV), v.to(DEV), torch.tensor(lengths, dtype=torch.int32, device=DEV), out,
                        window, sinks)
    ref, vmax = R.window_attention(q.float().numpy(), k.float().numpy(), v.float().numpy(), lengths, window, sinks)
    got = out.cpu().double().numpy()
    for b, L in enumerate(lengths):
        assert np.all(got[b, :, L:] == -7.25)               # rows behind the sequence are left as they were
        bound = (1 + 2.0 ** -6) * 2.0 ** -8 * (np.abs(ref[b, :, :L]) + vmax[b, :, :L, None])
        err = np.abs(got[b, :, :L] - ref[b, :, :L])
        assert np.all(err <= bound), float((err / bound).max())
    return out


@pytest.mark.parametrize("Hq,Hkv,d", [(2, 1, 64), (3, 3, 96), (4, 2, 128), (2, 2, 8), (7, 1, 72)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (5, 0), (100, 4), (127, 0), (128, 128), (129, 3),
                                          (256, 300), (333, 7), (2000, 4)])
def test_window_matches_reference(Hq, Hkv, d, window, sinks):
    lengths = [700, 0, 1, 129, 384, 641]
    op = DropKV(6, Hq, Hkv, d, 700, 1, out_rows=1, device=DEV)
    _check(op, *_inputs(6, Hq, Hkv, d, 700, lengths, seed=d), lengths, window, sinks)
    assert op.check() == 0


@pytest.mark.parametrize("n", [1, 2, 127, 128, 129, 255, 256, 257])
def test_window_short_prompts(n):
    op = DropKV(1, 2, 1, 64, n, 1, out_rows=1, device=DEV)
    for window, sinks in ((0, 0), (1, 0), (3, 2), (128, 1), (n, 0), (2 ** 31 - 1, 2 ** 31 - 1)):
        _check(op, *_inputs(1, 2, 1, 64, n, [n], seed=n), [n], window, sinks)


def test_without_a_window_it_is_the_prefill_attention():
    op = DropKV(2, 4, 2, 128, 900, 1, out_rows=1, device=DEV)
    q, k, v = (t.to(DEV) for t in _inputs(2, 4, 2, 128, 900, [900, 900]))
    a, b, c = (torch.zeros_like(q) for _ in range(3))
    op.prefill_attention(q, k, v, None, a)
    op.window_attention(q, k, v, None, b, 0)
    op.window_attention(q, k, v, None, c, 900, 5)
    assert torch.equal(b, c)
    assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -7 * float(v.float().abs().max())


def test_first_tokens_far_from_the_window():
    """Large first keys (an attention sink) that every row keeps, and the rows'
    own window far behind them."""
    op = DropKV(1, 2, 1, 128, 2100, 1, out_rows=1, device=DEV)
    q, k, v = _inputs(1, 2, 1, 128, 2100, [2100])
    k[0, 0, 0] = q[0, 0, :2000].float().mean(0).bfloat16() * 40
    v[0, 0, 0] = 3.0
    _check(op, q, k, v, [2100], 64, 1)
    _check(op, q, k, v, [2100], 64, 0)


def test_refusals_and_flags():
    op = DropKV(2, 4, 2, 64, 256, 1, out_rows=1, device=DEV)
    q, k, v = (t.to(DEV) for t in _inputs(2, 4, 2, 64, 256, [256, 256]))
    out = torch.zeros_like(q)
    for args in ((q, k, v, None, q, 5, 0), (q, k, v, None, out, -1, 0), (q, k, v, None, out, 5, -1)):
        with pytest.raises(DropKVError) as e:
            op.window_attention(*args)
        assert e.value.code == 1
    for args in ((q.float(), k, v, None, out, 5), (q[:1], k, v, None, out, 5), (q, k.cpu(), v, None, out, 5),
                 (q, k, v, torch.zeros(2, dtype=torch.int64, device=DEV), out, 5)):
        with pytest.raises(ValueError):
            op.window_attention(*args)
    with pytest.raises(ValueError):
        op.window_attention(q, k, v, None, out, 1 << 33)
    op.window_attention(q, k, v, torch.zeros(2, dtype=torch.int32, device=DEV), out, 5)
    assert B.kvcache_read_status(op.status) == (0, 0) and torch.all(out == 0)
    op.window_attention(q, k, v, torch.tensor([257, -1], dtype=torch.int32, device=DEV), out, 5)
    assert B.kvcache_read_status(op.status) == (7, B.FLAG_BAD_LENGTH)
    assert torch.all(out == 0)


def test_window_on_another_stream_and_in_a_graph():
    op = DropKV(1, 4, 2, 128, 1000, 1, out_rows=1, device=DEV)
    q, k, v = (t.to(DEV) for t in _inputs(1, 4, 2, 128, 1000, [1000]))
    want, out = torch.zeros_like(q), torch.zeros_like(q)
    op.window_attention(q, k, v, None, want, 300, 4)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    op.window_attention(q, k, v, None, out, 300, 4, stream=st)
    st.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.window_attention(q, k, v, None, out, 300, 4)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("lengths,window,sinks", [
    ([128, 1, 257, 384, 640, 129, 100, 0, 896], 0, 0),      # odd counts of tiles: items of one query tile
    ([128, 1, 257, 384, 640, 129, 100, 0, 896], 200, 5),
    ([4096, 3968], 2048, 4), ([4096, 3968], 600, 200), ([4096, 3968], 0, 0)])
def test_many_items_a_block_again_and_again(lengths, window, sinks):
    """Blocks that walk many items one after another, pass upon pass: the same
    bits each time and no wait given up.  (A warp that looked at a barrier two
    phases late would wait for its own work.)"""
    B_, n = len(lengths), max(lengths)
    H = 160 if n < 1000 else 32
    op = DropKV(B_, H, 4, 128, n, 1, out_rows=1, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(5)
    q, k, v = (torch.randn(B_, h, n, 128, generator=g, device=DEV).bfloat16() for h in (H, 4, 4))
    lens = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    want, out = torch.zeros_like(q), torch.zeros_like(q)
    op.window_attention(q, k, v, lens, want, window, sinks)
    for _ in range(20):
        op.window_attention(q, k, v, lens, out, window, sinks)
        assert torch.equal(out, want)
    assert op.check() == 0


@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 3), (300, 200)])
def test_more_sequences_than_a_warp_has_lanes(window, sinks):
    """The order of the items goes by chunks of 32 sequences: lengths of every
    kind in each, none at all in one, and lengths that cannot be served."""
    lengths = [(37 * b * b) % 401 if b % 5 else 400 for b in range(32)] + [0] * 32 + [400, 1, 129, 0, 256, 257, 383]
    op = DropKV(len(lengths), 2, 1, 16, 400, 1, out_rows=1, device=DEV)
    q, k, v = _inputs(len(lengths), 2, 1, 16, 400, lengths, seed=4)
    want = _check(op, q, k, v, lengths, window, sinks)
    assert op.check() == 0
    bad = list(lengths)
    bad[3], bad[66] = 401, -5                     # left out; the others as they were
    out = torch.full_like(want, -7.25)
    op.window_attention(q.to(DEV), k.to(DEV), v.to(DEV), torch.tensor(bad, dtype=torch.int32, device=DEV), out, window,
                        sinks)
    assert B.kvcache_read_status(op.status)[1] == B.FLAG_BAD_LENGTH
    for b in range(len(lengths)):
        assert torch.equal(out[b], want[b]) if b not in (3, 66) else torch.all(out[b] == -7.25)


def test_items_longer_than_a_waits_limit():
    """In the build whose waits end after 10 ms: 2^21 causal rows, whose last
    query tiles take some 20 ms each, are no timeout, and the bytes are those
    of the library."""
    n = 1 << 21
    g = torch.Generator(device=DEV).manual_seed(2)
    q, k, v = (torch.randn(1, 1, n, 8, generator=g, device=DEV).bfloat16() for _ in range(3))
    want, out = torch.zeros_like(q), torch.zeros_like(q)
    op = DropKV(1, 1, 1, 8, n, 1, out_rows=1, device=DEV)
    op.window_attention(q, k, v, None, want, 0)
    assert op.check() == 0
    hooks = _build.build_library(variant="test_hooks")
    with B.use_library(hooks):
        op.window_attention(q, k, v, None, out, 0)
        assert B.kvcache_read_status(op.status) == (0, 0)
    assert torch.equal(out, want)
