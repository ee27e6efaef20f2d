"""Failure detection in the shared attention, without a GPU fault: the test
build of the library (waits of 10 ms) leaves one load of one CTA out.  The waits
for it run out, every role of the CTA leaves its loop, copies and MMAs in flight
are waited for, the tensor memory is released, the status reads
DROPKV_ERR_TIMEOUT; heads that the CTA had no part in are whole, and the next
calls on the same context are clean."""
import os
import subprocess
import time

import pytest
import torch

from kv_cache_eviction_dropkv_gb300 import _binding as B, _build


def test_product_library_exports_no_hook():
    hooks = B.declared_functions(os.path.join(_build.INCLUDE, "kvcache_step_test_hooks.h"))
    assert hooks == ["kvcache_test_skip_shared_load"]
    out = subprocess.run(["nm", "-D", "--defined-only", _build.build_library()], capture_output=True, text=True,
                         check=True).stdout
    assert hooks[0] not in out


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("members", [3, 80])
@pytest.mark.parametrize("load", [0, 1, 2, 3])
def test_a_load_that_never_comes(d, members, load):
    """Four KV heads of 32 tiles, two to a CTA: CTA 5 has tiles of head 0 alone.
    3 and 80 members with 4 rows each: both kinds of units."""
    from tests.test_gpu_shared import forked, ints, queries

    c, seqs, starts = forked([4096], [[1 + i % 30 for i in range(members)]], 4, 4, d, 128, seed=3)
    q, who, groups = queries(members, 16, 1, d, 3), ints(seqs), ints(starts)
    want, out = torch.empty_like(q), torch.empty_like(q)
    c.shared_attention(0, q, want, groups, seqs=who, least=0)
    assert c.check() == 0
    with B.use_library(_build.build_library(variant="test_hooks")) as L:
        assert L.kvcache_test_skip_shared_load(5, load) == 0
        try:
            torch.cuda.synchronize()
            t0 = time.perf_counter()
            c.shared_attention(0, q, out.fill_(-7.25), groups, seqs=who, least=0)
            code, flags = B.kvcache_read_status(c.status)
            secs = time.perf_counter() - t0
        finally:
            assert L.kvcache_test_skip_shared_load(-1, -1) == 0
        assert (code, flags) == (8, B.FLAG_TIMEOUT)
        assert secs < 0.5, secs
        assert torch.equal(out[:, 4:], want[:, 4:])
        for _ in range(2):
            c.reset_status()
            c.shared_attention(0, q, out.fill_(-7.25), groups, seqs=who, least=0)
            assert c.check() == 0 and torch.equal(out, want)
    c.shared_attention(0, q, out.fill_(-7.25), groups, seqs=who, least=0)
    assert c.check() == 0 and torch.equal(out, want)
