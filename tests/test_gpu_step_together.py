"""The step's operators as a serving program uses them around an eviction: a
prompt's packed projection normed and turned, its attention with the eviction
fused in, the kept rows stored, samples forked from it, decode steps that store
their rotated tokens and attend over the shared pages, and one sample read back,
scored again and evicted.  Each step is held to the bounds of its own tests."""
import numpy as np
import pytest
import torch

import oracle
from kv_cache_eviction_dropkv_gb300 import DropKV, PagedCache, Rotary
from tests._parity import check_scores
from tests.test_gpu_paged import DEV, draw_rows, ints
from tests.test_gpu_shared import check as check_shared, noise
from tests.test_gpu_step import near, reference, weights

pytestmark = pytest.mark.gpu


def projected(n, rows, Hq, Hkv, d, seed):
    """A layer's projection, one row per token, as views of heads first."""
    x = draw_rows(n, rows, Hq + 2 * Hkv, d, seed, 0.3).to(DEV)
    return tuple(t.transpose(1, 2) for t in x.split((Hq, Hkv, Hkv), 2))


@pytest.mark.parametrize("code,layout,kind,kw", [("e4m3", "half", "bands", dict(factor=8.0, original=64)),
                                                 ("int8", "interleaved", "yarn", dict(factor=4.0, original=128))])
def test_prompt_samples_decode_and_rescoring(code, layout, kind, kw):
    Hq, Hkv, d, n, w, page, samples, base = 8, 2, 128, 610, 8, 32, 5, 10000.0
    dims = 128 if layout == "half" else 64
    qw, kw_ = weights(d, 1), weights(d, 2)
    rotary = Rotary(d, dims=dims, base=base, layout=layout, scaling=dict(kind=kind, **kw), q_norm=qw, k_norm=kw_, device=DEV)
    turn = lambda x, weight, at: reference(x, weight, at, d, dims, layout, base, kind, kw)
    q, k, v = projected(1, n, Hq, Hkv, d, 3)
    q_all, k_all = torch.empty(1, Hq, n, d, dtype=torch.bfloat16, device=DEV), torch.empty(1, Hkv, n, d, dtype=torch.bfloat16, device=DEV)
    v_all = v.contiguous()
    rotary.apply(q, k, q_all, k_all)
    near(q_all, *turn(q, qw, np.arange(n)[None])), near(k_all, *turn(k, kw_, np.arange(n)[None]))

    op = DropKV(1, Hq, Hkv, d, n, w, device=DEV)
    out, lengths, evict = torch.empty_like(q_all), ints([n]), ints([200])
    op.run_prefill(q_all, k_all, v_all, lengths, evict, out)
    assert op.check() == 0 and op.kept_len.tolist() == [410]
    ref = oracle.prefill_attention(q_all.cpu(), k_all.cpu(), v_all.cpu(), np.array([n]))
    top = float(v_all.abs().max())
    assert np.all(np.abs(out.cpu().double().numpy() - ref) <= 2.0 ** -8 * (np.abs(ref) + top) * (1 + 2.0 ** -6))

    # the kept rows are stored once and sampled from
    c = PagedCache(1 + samples, Hkv, d, 60, page, 20, 1, code, Hq=Hq, T=2, device=DEV, groups=2)
    noise(c, 5)
    c.reserve(op.kept_len, seqs=ints([0]))
    c.store(0, op.k_out, op.v_out, op.kept_len, seqs=ints([0]))
    who = list(range(1, 1 + samples))
    c.fork(ints([0] * samples), ints(who))
    for step, T in enumerate((1, 1, 2, 1)):
        at = n + sum((1, 1, 2, 1)[:step])                         # positions go on where the prompt ended, slots do not
        c.reserve(ints([T] * samples), seqs=ints(who))
        q, k, v = projected(samples, T, Hq, Hkv, d, 20 + step)
        q_out = torch.empty(samples, Hq, T, d, dtype=torch.bfloat16, device=DEV)
        c.store_rotated(0, rotary, q, k, v, q_out, positions=ints([at] * samples), seqs=ints(who))
        here = np.tile(at + np.arange(T), (samples, 1))
        near(q_out, *turn(q, qw, here))
        # what the cache holds of the tokens is within half a code's step of the formula
        want, bound = turn(k, kw_, here)
        got, got_v = (torch.empty(samples, Hkv, T, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        c.read(0, got, got_v, starts=c.length[1:] - T, counts=ints([T] * samples), seqs=ints(who))
        last = c.table[who, ((c.length[1:] - 1) // page).long()].long()
        scale = c.k_scale[0, last].double().cpu().numpy()         # [samples][Hkv], the page of the last token
        half = 0.5 * scale[..., None, None] if code == "int8" else 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * scale[..., None, None]
        if step in (0, 1, 3):                                     # (one token: one page)
            err = np.abs(got.cpu().double().numpy() - want)
            assert np.all(err <= (half + bound) * (1 + 2.0 ** -4) + 2.0 ** -8 * np.abs(want))
        check_shared(c, q_out, who, [0, samples])
        assert c.check() == 0 and rotary.check() == 0

    # one sample is read back, scored by the window of its newest queries, and evicted
    mine, m = who[2], int(c.length[who[2]])
    k_back, v_back = (torch.zeros(1, Hkv, m, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    c.read(0, k_back, v_back, seqs=ints([mine]))
    again = DropKV(1, Hq, Hkv, d, m, w, device=DEV)
    window = q_all[:, :, -w:].contiguous()
    again.run(window, k_back, v_back, ints([m]), ints([m // 2]))
    assert again.check() == 0
    ref = oracle.run_path(window.cpu(), k_back.cpu(), v_back.cpu(), torch.tensor([m], dtype=torch.int32),
                          torch.tensor([m // 2], dtype=torch.int32), 5, w)
    check_scores(again.scores.cpu().numpy(), ref["final"], np.array([m]), "read back")
    assert again.kept_len.tolist() == ref["kept_len"].tolist() == [m - m // 2]
    c.compact(again.kept_idx.reshape(1, 1, Hkv, -1), again.kept_len, ints([mine]))
    assert int(c.length[mine]) == m - m // 2 and c.check() == 0
    # the others still share the prompt's pages, the evicted one shares nothing and takes no part
    q1 = draw_rows(samples, Hq, 1, d, 60, 0.3).to(DEV)
    check_shared(c, q1, who, [0, samples])
    check_shared(c, q1, [who[0], who[1], who[3], who[4], mine], [0, 4, 5])
    c.free(ints([0] + who))
    assert int(c.refs.abs().sum()) == 0 and c.check() == 0
