"""The operators as a serving loop uses them: a prompt's attention with the
eviction fused in, the kept rows into the 8-bit cache, decode steps, forks of
the sequence, an eviction of one branch, a windowed prompt beside it.  Every
step is compared with the plain reference in 64 bits, with the bounds of the
operators' own tests."""
import numpy as np
import pytest
import torch

from kv_cache_eviction_dropkv_gb300 import DropKV, PagedCache, synth
from tests import _paged as R
from tests.test_gpu_paged import both, check_attention, draw_rows, ints, same_pool, same_state

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0) if torch.cuda.is_available() else None


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_prompt_eviction_decode_fork_evict_free(code):
    wl = synth.make_workload("qwen_gqa7_b4_ragged_n64k", n_max=700, seed=5)
    s = wl.spec
    rng = np.random.default_rng(1)
    q_all = rng.standard_normal((s.B, s.Hq, s.n_max, s.d)).astype(np.float32)
    for b in range(s.B):
        nb = int(wl.lengths[b])
        q_all[b, :, nb - s.w:nb] = wl.q[b].float().numpy()
    op = DropKV(s.B, s.Hq, s.Hkv, s.d, s.n_max, s.w, s.pool_kernel, s.protect, device=DEV)
    out = torch.zeros(s.B, s.Hq, s.n_max, s.d, dtype=torch.bfloat16, device=DEV)
    op.run_prefill(synth.bf16_round(q_all).to(DEV), wl.k.to(DEV), wl.v.to(DEV), wl.lengths.to(DEV), wl.evict_k.to(DEV), out)
    op.check()
    kept = op.kept_len.tolist()
    assert kept == wl.kept_len().tolist()

    seqs, page, M = 3 * s.B, 32, 8
    c = PagedCache(seqs, s.Hkv, s.d, 96, page, M, 1, code, Hq=s.Hq, T=2, device=DEV)
    r = R.RefCache(seqs, s.Hkv, s.d, 96, page, M, 1, code)
    # the kept rows move in: the compacted rows and counts are store()'s arguments as they are
    c.reserve(op.kept_len)
    r.reserve(kept)
    c.store(0, op.k_out, op.v_out, op.kept_len)
    rows = max(kept)
    r.store(0, op.k_out[:, :, :rows].float().cpu().numpy(), op.v_out[:, :, :rows].float().cpu().numpy(), kept)
    same_state(c, r)
    same_pool(c, r)

    def step(who, T, seed, **kw):
        both(c, r, "reserve", [T] * len(who), seqs=who)
        k, v, q = (draw_rows(len(who), h, T, s.d, seed + i, spread=0.3) for i, h in enumerate((s.Hkv, s.Hkv, s.Hq)))
        both(c, r, "store", 0, k, v, [T] * len(who), seqs=who)
        check_attention(c, r, q, seqs=who, **kw)

    first = list(range(s.B))
    for i in range(3):
        step(first, 1, 100 + 10 * i)
    step(first, 2, 200, window=17, sinks=2)
    # parallel samples of each sequence; the first ones go on, too
    both(c, r, "fork", first + first, list(range(s.B, 3 * s.B)))
    everyone = list(range(3 * s.B))
    for i in range(2):
        step(everyone, 1, 300 + 10 * i)
    same_state(c, r)
    # one branch of each is evicted again, with the scores of the layer
    branch = list(range(s.B, 2 * s.B))
    lengths = [r.length[x] for x in branch]
    left = [x - 5 for x in lengths]
    idx = np.zeros((1, s.B, s.Hkv, max(left)), dtype=np.int64)
    for i, (n, m) in enumerate(zip(lengths, left)):
        for h in range(s.Hkv):
            idx[0, i, h, :m] = np.sort(rng.permutation(n)[:m])
    c.compact(ints(idx.tolist()), ints(left), ints(branch))
    r.compact(idx.tolist(), left, branch)
    same_state(c, r)
    step(everyone, 1, 400)
    step(branch, 2, 410, window=9, sinks=1)
    c.free(ints(first))
    r.free(first)
    step(branch + list(range(2 * s.B, 3 * s.B)), 1, 420)
    same_state(c, r)
    same_pool(c, r)
    c.free(ints(everyone))
    assert int(c.refs.abs().sum()) == 0 and c.check() == 0


def test_windowed_prompt_then_windowed_decode():
    """The positional baseline end to end: the prompt with a sliding window and
    kept first tokens, its rows stored, decode steps with the same window."""
    Hq, Hkv, d, n, W, S = 8, 2, 128, 500, 130, 4
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(1, h, n, d, generator=g).bfloat16() for h in (Hq, Hkv, Hkv))
    op = DropKV(1, Hq, Hkv, d, n, 1, out_rows=1, device=DEV)
    out = torch.zeros(1, Hq, n, d, dtype=torch.bfloat16, device=DEV)
    op.window_attention(q.to(DEV), k.to(DEV), v.to(DEV), None, out, W, S)
    ref, vmax = R.window_attention(q.float().numpy(), k.float().numpy(), v.float().numpy(), [n], W, S)
    err = np.abs(out.cpu().double().numpy() - ref)
    assert np.all(err <= (1 + 2.0 ** -6) * 2.0 ** -8 * (np.abs(ref) + vmax[..., None]))
    c = PagedCache(1, Hkv, d, 20, 64, 10, Hq=Hq, device=DEV)
    r = R.RefCache(1, Hkv, d, 20, 64, 10, 1, "e4m3")
    both(c, r, "reserve", [n])
    both(c, r, "store", 0, k, v)
    for i in range(3):
        both(c, r, "reserve", [1])
        k1, v1, q1 = (draw_rows(1, h, 1, d, 50 + 3 * i + j, spread=0.2) for j, h in enumerate((Hkv, Hkv, Hq)))
        both(c, r, "store", 0, k1, v1)
        check_attention(c, r, q1, window=W, sinks=S)
    assert c.check() == 0 and op.check() == 0
