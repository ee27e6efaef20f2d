"""Failure detection in the windowed prompt attention, without a GPU fault: the
test build of the library (waits of 10 ms) leaves one K/V pair of one CTA out.
The waits for it run out, every role of the CTA leaves its loop, copies and
MMAs in flight are waited for, the tensor memory is released, the status reads
DROPKV_ERR_TIMEOUT; rows are the library's or were not written, the other CTAs'
items are whole, and the next calls on the same context are clean."""
import os
import subprocess
import time

import pytest
import torch

from kv_cache_eviction_dropkv_gb300 import DropKV, _binding as B, _build

DEV = torch.device("cuda", 0) if torch.cuda.is_available() else None


def test_product_library_exports_no_hook():
    hooks = B.declared_functions(os.path.join(_build.INCLUDE, "kvcache_test_hooks.h"))
    assert hooks == ["kvcache_test_skip_window_pair"]
    out = subprocess.run(["nm", "-D", "--defined-only", _build.build_library()], capture_output=True, text=True,
                         check=True).stdout
    assert hooks[0] not in out


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 3)])
@pytest.mark.parametrize("pair,lost", [(0, 2), (1, 2), (2, 2), (3, 1), (4, 1)])
def test_a_pair_that_never_comes(d, window, sinks, pair, lost):
    """Two items for each CTA, two key tiles each: pairs 0 and 1 are the first
    item's, pair 2 the last V of the first with the first K of the second,
    pair 4 the last V alone.  lost: items that the CTA cannot finish."""
    Hq, n = 2 * torch.cuda.get_device_properties(0).multi_processor_count, 256
    g = torch.Generator(device=DEV).manual_seed(3)
    q, k, v = (torch.randn(1, h, n, d, generator=g, device=DEV).bfloat16() for h in (Hq, Hq, Hq))
    op = DropKV(1, Hq, Hq, d, n, 1, out_rows=1, device=DEV)
    want = torch.zeros_like(q)
    op.window_attention(q, k, v, None, want, window, sinks)
    assert op.check() == 0
    with B.use_library(_build.build_library(variant="test_hooks")) as L:
        out = torch.full_like(q, -7.25)
        assert L.kvcache_test_skip_window_pair(5, pair) == 0
        try:
            torch.cuda.synchronize()
            t0 = time.perf_counter()
            op.window_attention(q, k, v, None, out, window, sinks)
            code, flags = B.kvcache_read_status(op.status)
            secs = time.perf_counter() - t0
        finally:
            assert L.kvcache_test_skip_window_pair(-1, -1) == 0
        assert (code, flags) == (8, B.FLAG_TIMEOUT)
        assert secs < 0.5, secs
        whole = (out == want).all(-1)
        assert torch.all(whole | (out == -7.25).all(-1))
        assert int((~whole).any(-1).sum()) == lost
        for _ in range(2):
            op.reset_status()
            out.fill_(-7.25)
            op.window_attention(q, k, v, None, out, window, sinks)
            assert op.check() == 0 and torch.equal(out, want)
    out.fill_(-7.25)
    op.window_attention(q, k, v, None, out, window, sinks)
    assert op.check() == 0 and torch.equal(out, want)
