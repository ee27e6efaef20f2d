"""Refusals of kvcache_run's own fields, without a GPU: addresses are never followed."""
import ctypes

import pytest

from kv_cache_eviction_dropkv_gb300 import _binding as B, _build
from tests.test_kvcache_boundary import A, INVALID, buffers, shape


@pytest.fixture(scope="module", autouse=True)
def _library():
    _build.build_library()


def test_where_a_reservations_grants_go():
    s, b = shape(), buffers()
    run = lambda out, n, extra=A: B.lib().kvcache_run(B.kvcache_call.pack(
        ctypes.addressof(s), ctypes.addressof(b), A, 1 << 30, A, 0, 0, extra, 0, 0, out, B.RESERVE_GRANTED, 0, n,
        0, 0, 0, 0))
    assert run(A + 2, 2) == INVALID and run(A + 1, 0) == INVALID and run(0, 2) == INVALID
    assert run(A + 4, 2, extra=0) == INVALID and run(A + 4, 0) == 0
