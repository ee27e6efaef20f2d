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


def test_yarn_ramps_the_wrong_way_round_are_refused():
    """A bound of the slow pairs above that of the fast ones, as "bands" refuses it."""
    plan = dict(kind="yarn", factor=8.0, original=4096)
    for bad in (dict(fast=1.0, slow=32.0), dict(slow=33.0), dict(fast=0.5)):
        with pytest.raises(ValueError):
            rotary.frequencies(64, 10000.0, {**plan, **bad})
    for good in (dict(fast=2.0, slow=2.0), dict(fast=None, slow=None), dict(fast=33.0, slow=31.0)):
        rotary.frequencies(64, 10000.0, {**plan, **good})
