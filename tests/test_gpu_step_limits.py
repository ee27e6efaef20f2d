"""Rotations at their limits: tensors without heads, what the sine and cosine
are off by, elements and an eps near the ends of fp32."""
import numpy as np
import pytest
import torch

from kv_cache_eviction_dropkv_gb300 import Rotary
from tests.test_gpu_paged import DEV
from tests.test_gpu_step import rows, weights

gpu = pytest.mark.gpu
pytestmark = gpu


def within(got, want, off):
    """got (bf16) is the rounding of a number that is `off` from want at most."""
    # (fp32 in between is off by half a step of 2^-24 more, for numbers up to 1)
    lo, hi = (torch.from_numpy((want + s * (off + 2.0 ** -25)).astype(np.float32)).bfloat16() for s in (-1, 1))
    return bool(((lo <= got) & (got <= hi)).all())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_sine_and_cosine_are_off_by_a_last_place_of_fp32(layout):
    """2^-23, at any position.  Pairs (1, 0) become (cos, sin) without another
    rounding but the last; of 2^23 results some thousands lie within 2^-20 of a
    border between two bf16 numbers, so that a wrong place shows."""
    d, n = 128, 1 << 16
    plan = Rotary(d, base=1000003.0, layout=layout, device=DEV)
    at = np.random.default_rng(7).integers(-2 ** 31, 2 ** 31, n)
    at[:4] = -2 ** 31, 2 ** 31 - 1, 0, -1
    a, b = (slice(0, d // 2), slice(d // 2, d)) if layout == "half" else (slice(0, d, 2), slice(1, d, 2))
    q = torch.zeros(1, 1, n, d, dtype=torch.bfloat16, device=DEV)
    q[..., a] = 1.0
    out = torch.empty_like(q)
    plan.apply(q, None, out, None, positions=torch.from_numpy(at).to(torch.int32).to(DEV)[None])
    assert plan.check() == 0
    turns = at.astype(np.int64).view(np.uint64)[:, None] * plan.turns.cpu().numpy().view(np.uint64)[None]   # (modulo 2^64)
    angle = 2 * np.pi * (turns.astype(np.float64) * 2.0 ** -64)
    for got, want in ((out[0, 0][:, a].cpu(), np.cos(angle)), (out[0, 0][:, b].cpu(), np.sin(angle))):
        assert within(got, want, 2.0 ** -23)
        assert not within(got, want + 2.0 ** -20, 2.0 ** -23)


def test_a_tensor_without_heads_leaves_the_other_one():
    """As in store_rotated(): no heads are no queries, or no keys."""
    plan = Rotary(64, q_norm=weights(64, 1), k_norm=weights(64, 2), device=DEV)
    q, k = rows(2, 6, 9, 64, 1), rows(2, 2, 9, 64, 2)
    q_out, k_out = torch.empty_like(q), torch.empty_like(k)
    plan.apply(q, k, q_out, k_out)
    for none in (q[:, :0], None):
        got = torch.full_like(k, 7.0)
        plan.apply(none, k, none, got)
        assert torch.equal(got, k_out)
    for none in (k[:, :0], None):
        got = torch.full_like(q, 7.0)
        plan.apply(q, none, got, none)
        assert torch.equal(got, q_out)
    plan.apply(q[:, :0], k[:, :0], q[:, :0], k[:, :0])
    plan.apply(q[:, :0], k, None, got := torch.empty_like(k))
    assert torch.equal(got, k_out) and plan.check() == 0


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("x,eps", [(2.0 ** 64, 2.0 ** 127), (2.0 ** 60, 3.4028234e38), (2.0 ** 64, 1e-6), (3.3e38, 1e38),
                                   (1.0, 3.4028234e38), (2.0 ** -60, 1e-30)])
def test_norms_where_squares_or_eps_reach_the_end_of_fp32(layout, x, eps):
    """x / sqrt(mean x^2 + eps) of rows of one magnitude and of rows with a few
    large elements.  Bound: the tests' of a norm, 2^-8 + 2^-19 of the value, and
    bf16's smallest half step."""
    plan = Rotary(64, dims=0, layout=layout, q_norm=torch.ones(64), eps=eps, device=DEV)
    q = rows(2, 3, 5, 64, 1).sign() * x
    q[:, 1, :, 9:] *= 2.0 ** -10
    out = torch.empty_like(q)
    plan.apply(q, None, out, None)
    y = q.cpu().double().numpy()
    want = y / np.sqrt((y * y).mean(-1, keepdims=True) + float(np.float32(eps)))
    assert np.all(np.abs(out.cpu().double().numpy() - want) <= (2.0 ** -8 + 2.0 ** -19) * np.abs(want) + 2.0 ** -134)
