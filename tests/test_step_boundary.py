"""Host-side refusals of include/kvcache_step.h, and the table of frequencies,
without a GPU: addresses are never followed."""
import ctypes
import math

import numpy as np
import pytest
import torch

from kv_cache_eviction_dropkv_gb300 import _binding as B, _build, rotary
from tests.test_kvcache_boundary import A, INVALID, UNSUPPORTED, WORKSPACE, buffers, shape

FAR = A + (1 << 30)                           # away from everything else


@pytest.fixture(scope="module", autouse=True)
def _library():
    _build.build_library()


def plan(turns=A, q_norm=A, k_norm=None, d=64, dims=64, layout=0, eps=1e-6, amplitude=1.0):
    return B.kvcache_rotary(turns, q_norm, k_norm, d, dims, layout, eps, amplitude)


def rotate(p=None, q=(A, 4 * 3 * 64, 3 * 64, 64), k=(A + (1 << 20), 2 * 3 * 64, 3 * 64, 64), q_out=FAR, k_out=FAR + (1 << 24),
           positions=A, lengths=A, status=A, Bn=2, Hq=4, Hkv=2, n=3, kind=0):
    p = plan() if p is None else p
    return B.lib().kvcache_rotate(B.rotate_call.pack(ctypes.addressof(p), *q, *k, q_out, k_out, positions, lengths, status,
                                                     0, Bn, Hq, Hkv, n, kind))


def store(p=None, q=(A, 4 * 3 * 64, 3 * 64, 64), k=(A, 2 * 3 * 64, 3 * 64, 64), v=(A, 2 * 3 * 64, 3 * 64, 64), q_out=FAR,
          s=None, b=None, seqs=0, counts=0, positions=0, status=A, layer=0, n=2, Hq=4, rows=3, kind=0):
    p, s, b = plan() if p is None else p, shape() if s is None else s, buffers() if b is None else b
    return B.lib().kvcache_rotate_store(B.rotate_store_call.pack(
        ctypes.addressof(s), ctypes.addressof(b), ctypes.addressof(p), *q, *k, *v, q_out, seqs, counts, positions, status, 0,
        layer, n, Hq, rows, kind))


def read(s=None, b=None, seqs=0, starts=0, counts=0, k=A, v=FAR, status=A, layer=0, n=2, rows=3):
    s, b = shape() if s is None else s, buffers() if b is None else b
    return B.lib().kvcache_read(B.read_call.pack(ctypes.addressof(s), ctypes.addressof(b), seqs, starts, counts, k, v,
                                                 status, 0, layer, n, rows))


def shared(s=None, b=None, seqs=0, groups=A, q=A, out=FAR, ws=A, wsb=1 << 40, status=A, layer=0, n=2, Hq=4, T=1, G=1, least=0):
    s, b = shape() if s is None else s, buffers() if b is None else b
    return B.lib().kvcache_shared_attention(B.shared_attention_call.pack(
        ctypes.addressof(s), ctypes.addressof(b), seqs, groups, q, out, ws, wsb, status, 0, least, layer, n, Hq, T, G))


def test_every_declared_symbol_is_exported_and_bound():
    lib = B.lib()
    names = B.declared_functions(_build.INCLUDE + "/kvcache_step.h")
    assert len(names) == 5
    for name in names:
        assert hasattr(lib, name) and getattr(lib, name).argtypes is not None, name
    for name in B.STEP_CALLS:
        assert getattr(lib, name)(None) == INVALID


def test_records_have_the_size_of_the_structures():
    # pointers and 64-bit fields first, then 32-bit ones: no padding but at the end
    rows = 8 + 3 * 8
    up = lambda x: (x + 7) // 8 * 8
    assert B.rotate_call.size == 8 + 2 * rows + 6 * 8 + up(5 * 4)
    assert B.rotate_store_call.size == 3 * 8 + 3 * rows + 6 * 8 + up(5 * 4)
    assert B.read_call.size == 9 * 8 + up(3 * 4)
    assert B.shared_attention_call.size == 11 * 8 + up(5 * 4)
    assert ctypes.sizeof(B.kvcache_rotary) == 3 * 8 + up(5 * 4)


@pytest.mark.parametrize("kw,code", [
    (dict(d=0), INVALID), (dict(dims=-8), INVALID), (dict(dims=72), INVALID), (dict(layout=2), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID),
    (dict(amplitude=math.inf), INVALID), (dict(turns=None), INVALID), (dict(turns=A + 8), INVALID),
    (dict(q_norm=A + 4), INVALID), (dict(k_norm=A + 8), INVALID), (dict(d=60, dims=8), UNSUPPORTED),
    (dict(d=136, dims=8), UNSUPPORTED), (dict(dims=12), UNSUPPORTED)])
def test_plans_are_refused(kw, code):
    assert rotate(plan(**kw)) == code
    assert store(plan(**kw)) == code


def test_rotation_arguments():
    dense = (A, 4 * 3 * 64, 3 * 64, 64)
    assert [rotate(Bn=-1), rotate(n=-1), rotate(Hq=0), rotate(Hkv=0), rotate(status=0), rotate(status=A + 2),
            rotate(positions=A + 2), rotate(lengths=A + 1), rotate(kind=2), rotate(q_out=0), rotate(k_out=FAR + 8),
            rotate(q=(A + 8, 768, 192, 64)), rotate(q=(A, 768, 192, 60)), rotate(q=(A, -768, 192, 64)),
            rotate(k=(A, 1 << 50, 192, 64))] == [INVALID] * 15
    # outputs over inputs: q_out over q only where q is densely packed and the very same, and over nothing else
    assert rotate(q=(A, 4 * 3 * 64, 64, 4 * 64), q_out=A) == INVALID
    assert rotate(q=dense, q_out=A + 128) == INVALID
    assert rotate(q_out=A + (1 << 20)) == INVALID and rotate(k_out=A) == INVALID and rotate(k_out=FAR) == INVALID
    assert [rotate(Hq=65535), rotate(Bn=1 << 16, n=1 << 15)] == [UNSUPPORTED] * 2
    # nothing to do
    none = (0, 0, 0, 0)
    assert [rotate(Bn=0), rotate(n=0), rotate(q=none, k=none)] == [0] * 3


def test_store_arguments():
    assert [store(plan(d=128, dims=64)), store(rows=-1), store(Hq=0), store(kind=3), store(seqs=A + 2), store(counts=A + 1),
            store(positions=A + 2), store(status=0), store(layer=2), store(n=5), store(k=(0, 384, 192, 64)),
            store(v=(A, 384, 192, 4)), store(q_out=0), store(q_out=A), store(q_out=A + 64), store(q=(A + 2, 0, 0, 0)),
            store(b=buffers(table=None)), store(b=buffers(k=A + 8))] == [INVALID] * 18
    assert [store(s=shape(d=136)), store(s=shape(page=16)), store(rows=1 << 29, q=(A, 0, 0, 0))] == [UNSUPPORTED] * 3
    assert [store(n=0), store(rows=0)] == [0] * 2


def test_read_arguments():
    assert [read(rows=-1), read(n=5), read(layer=-1), read(status=0), read(k=0), read(v=A), read(v=FAR + 8),
            read(starts=A + 2), read(counts=A + 1), read(seqs=A + 2), read(b=buffers(length=None))] == [INVALID] * 11
    assert [read(n=0), read(rows=0)] == [0] * 2


def test_shared_attention_arguments():
    assert [shared(Hq=3), shared(Hq=0), shared(T=0), shared(G=0), shared(G=3), shared(groups=0), shared(groups=A + 2),
            shared(q=0), shared(out=A), shared(n=5), shared(layer=2), shared(status=0), shared(b=buffers(refs=None))
            ] == [INVALID] * 13
    assert [shared(T=1 << 20), shared(s=shape(page=96))] == [UNSUPPORTED] * 2
    assert shared(n=0) == 0


def test_workspace_sizes_are_refused():
    size = lambda s=None, n=2, Hq=4, T=1, G=1: B.kvcache_shared_workspace_size(shape() if s is None else s, n, Hq, T, G)
    assert [size(n=5), size(n=0), size(G=0), size(G=3), size(Hq=3), size(T=0), size(T=1 << 20), size(shape(d=60))] == [0] * 8


# ------------------------------------------------------------------ frequencies
def by_formula(dims, base, kind, **kw):
    i = np.arange(dims // 2, dtype=np.float64)
    if kind == "ntk":
        base = base * kw["factor"] ** (dims / (dims - 2))
    f = np.power(float(base), -2 * i / dims)
    if kind == "linear":
        return f / kw["factor"], 1.0
    if kind == "bands":
        turns = kw["original"] * f / (2 * np.pi)
        g = np.clip((turns - kw.get("low", 1)) / (kw.get("high", 4) - kw.get("low", 1)), 0, 1)
        return (1 - g) * f / kw["factor"] + g * f, 1.0
    if kind == "yarn":
        at = lambda r: dims * np.log(kw["original"] / (r * 2 * np.pi)) / (2 * np.log(base))
        lo, hi = max(np.floor(at(kw.get("fast", 32))), 0), min(np.ceil(at(kw.get("slow", 1))), dims - 1)
        g = 1 - np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
        return f / kw["factor"] * (1 - g) + f * g, 0.1 * np.log(kw["factor"]) + 1
    return f, 1.0


@pytest.mark.parametrize("dims", [8, 64, 96, 128])
@pytest.mark.parametrize("kind,kw", [(None, {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
                                     ("yarn", dict(factor=16.0, original=4096)),
                                     ("yarn", dict(factor=4.0, original=32768, fast=16.0, slow=2.0)),
                                     ("bands", dict(factor=8.0, original=8192)),
                                     ("bands", dict(factor=8.0, original=8192, low=2.0, high=32.0))])
def test_frequencies(dims, kind, kw):
    for base in (10000.0, 1e6):
        got, amplitude = rotary.frequencies(dims, base, dict(kind=kind, **kw) if kind else None)
        want, a = by_formula(dims, base, kind, **kw)
        np.testing.assert_allclose(got, want, rtol=1e-12)
        assert abs(amplitude - a) < 1e-12


def test_frequencies_are_refused():
    for bad in (dict(kind="linear"), dict(factor=2.0), dict(kind="other", factor=2.0), dict(kind="linear", factor=0.0),
                dict(kind="yarn", factor=2.0), dict(kind="linear", factor=2.0, original=5),
                dict(kind="bands", factor=2.0, original=4096, low=4.0, high=1.0), dict(kind="ntk", factor=math.nan)):
        with pytest.raises(ValueError):
            rotary.frequencies(64, 10000.0, bad)
    with pytest.raises(ValueError):
        rotary.frequencies(64, -1.0)
    assert rotary.frequencies(0) == ([], 1.0)


def test_plans_live_on_a_cuda_device():
    for kw in (dict(d=60), dict(d=136), dict(d=64, dims=72), dict(d=64, dims=4), dict(d=64, layout="other"),
               dict(d=64, eps=0.0), dict(d=64, device="cpu")):
        with pytest.raises(ValueError):
            rotary.Rotary(**{"device": "cuda", **kw})


def test_rows_of_views():
    x = torch.zeros(2, 5, 6, 64, dtype=torch.bfloat16)
    view = x.transpose(1, 2)
    assert B.rows_of("q", view, (2, 6, 5, 64), -1)[1:] == (5 * 6 * 64, 64, 6 * 64)
    wide = torch.zeros(2, 5, 6, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.rows_of("q", wide[..., ::2], (2, 5, 6, 64), -1)          # channels apart
    with pytest.raises(ValueError):
        B.rows_of("q", wide[..., 4:68], (2, 5, 6, 64), -1)         # rows off their boundary
    with pytest.raises(ValueError):
        B.rows_of("q", view.float(), (2, 6, 5, 64), -1)
    odd = torch.zeros(2 * 5 * 68, dtype=torch.bfloat16).as_strided((2, 1, 5, 64), (340, 3, 68, 1))
    with pytest.raises(ValueError):
        B.rows_of("q", odd, (2, 1, 5, 64), -1)
    one = torch.zeros(64, dtype=torch.bfloat16).as_strided((1, 1, 1, 64), (3, 5, 7, 1))
    B.rows_of("q", one, (1, 1, 1, 64), -1)                        # strides over single items are not used


def test_frequencies_without_a_ramp_are_refused():
    with pytest.raises(ValueError):                    # the ramp stands on powers of the base
        rotary.frequencies(64, 1.0, dict(kind="yarn", factor=2.0, original=4096))
    for kind in ("yarn", "bands"):
        with pytest.raises(ValueError):
            rotary.frequencies(64, 10000.0, dict(kind=kind, factor=2.0, original=None))
        with pytest.raises(ValueError):
            rotary.frequencies(64, 10000.0, dict(kind=kind, factor=None, original=4096))
    assert rotary.frequencies(64, 1.0, dict(kind="linear", factor=2.0)) == ([0.5] * 32, 1.0)
