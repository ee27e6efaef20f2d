"""Scalings of the frequencies at the ends of their ranges, without a GPU."""
import math

import pytest

from kv_cache_eviction_dropkv_gb300 import rotary


@pytest.mark.parametrize("factor,want", [(1e-6, 1.0), (0.5, 1.0), (1.0, 1.0), (1.5, 0.1 * math.log(1.5) + 1.0),
                                         (16.0, 0.1 * math.log(16.0) + 1.0)])
def test_yarn_amplitude(factor, want):
    """0.1 ln(factor) + 1 for a stretched context, 1 for one that is not."""
    scaling = dict(kind="yarn", factor=factor, original=4096)
    assert rotary.frequencies(64, 10000.0, scaling)[1] == pytest.approx(want, rel=1e-15)
    assert rotary.frequencies(64, 10000.0, dict(scaling, amplitude=0.75))[1] == 0.75
