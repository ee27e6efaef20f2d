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
