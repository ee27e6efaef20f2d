"""Host-side refusals of include/kvcache.h: they come before any CUDA call, so
they are checked without a GPU, with addresses that are never followed."""
import ctypes

import pytest

from kv_cache_eviction_dropkv_gb300 import _binding as B, _build
from tests import _paged as R

import numpy as np

INVALID, WORKSPACE, UNSUPPORTED = 1, 2, 6
GOOD = dict(layers=2, Hkv=2, d=64, page=64, pages=10, seqs=4, max_pages=5, code=0)
A = 1 << 20                                   # an aligned address


@pytest.fixture(scope="module", autouse=True)
def _library():
    _build.build_library()


def shape(**kw):
    return B.kvcache_shape(**{**GOOD, **kw})


def buffers(**kw):
    names = [f for f, _ in B.kvcache_buffers._fields_]
    return B.kvcache_buffers(**{**{n: A + 4096 * i for i, n in enumerate(names)}, **kw})


def calls(s, b, n=2, layer=0, ws=A, wsb=1 << 30, status=A):
    L, S, C = B.lib(), ctypes.byref(s), ctypes.byref(b)
    return [L.kvcache_reserve(S, C, None, n, A, ws, wsb, status, None),
            L.kvcache_store(S, C, layer, None, n, A, A, 3, None, status, None),
            L.kvcache_attention(S, C, layer, None, n, A, 4, 1, 0, 0, A + (1 << 20), ws, wsb, status, None),
            L.kvcache_fork(S, C, A, A, n, 1, ws, wsb, status, None),
            L.kvcache_compact(S, C, None, n, A, 8, A, ws, wsb, status, None),
            L.kvcache_free(S, C, A, n, status, None)]


def recorded(s, b, n=2, layer=0, ws=A, wsb=1 << 30, status=A):
    """The same calls through kvcache_run."""
    rec = lambda op, seqs, *rest: B.lib().kvcache_run(B.kvcache_call.pack(
        ctypes.addressof(s), ctypes.addressof(b), ws or 0, wsb, status or 0, 0, seqs, *rest[:4], op, layer, n, *rest[4:]))
    return [rec(B.RESERVE, 0, A, 0, 0, 0, 0, 0, 0, 0),
            rec(B.STORE, 0, A, A, 0, 0, 3, 0, 0, 0),
            rec(B.ATTENTION, 0, A, 0, 0, A + (1 << 20), 4, 1, 0, 0),
            rec(B.FORK, A, A, 0, 0, 0, 1, 0, 0, 0),
            rec(B.COMPACT, 0, A, A, 0, 0, 8, 0, 0, 0),
            rec(B.FREE, A, 0, 0, 0, 0, 0, 0, 0, 0)]


def test_records_make_the_same_calls():
    assert B.kvcache_call.size == 120
    s, b = shape(), buffers()
    for kw in (dict(n=0), dict(n=5), dict(n=-1), dict(layer=2, n=0), dict(wsb=64), dict(ws=None), dict(status=None)):
        if kw in (dict(wsb=64), dict(ws=None)):       # (the calls without a workspace would launch)
            got, want = recorded(s, b, n=0, **kw), calls(s, b, n=0, **kw)
        else:
            got, want = recorded(s, b, **kw), calls(s, b, **kw)
        assert got == want, kw
    rec = [ctypes.addressof(s), ctypes.addressof(b), A, 1 << 30, A, 0, 0, A, A, A, A + (1 << 20), 0, 0, 0, 4, 1, 0, 0]
    for op in (-1, 6):
        rec[11] = op
        assert B.lib().kvcache_run(B.kvcache_call.pack(*rec)) == INVALID
    assert B.lib().kvcache_run(None) == INVALID
    # arguments that are the call's own, each refused by the same call
    run = lambda op, in0, in1, in2, out, *arg: B.lib().kvcache_run(B.kvcache_call.pack(
        *rec[:7], in0, in1, in2, out, op, 0, 0, *arg))
    assert run(B.STORE, A, A, 0, 0, -1, 0, 0, 0) == INVALID and run(B.STORE, A, 0, 0, 0, 1, 0, 0, 0) == INVALID
    assert run(B.ATTENTION, A, 0, 0, A, 3, 1, 0, 0) == INVALID and run(B.ATTENTION, A, 0, 0, A, 4, 1, -1, 0) == INVALID
    assert run(B.ATTENTION, A, 0, 0, A, 4, 1, 0, -1) == INVALID and run(B.ATTENTION, A, 0, 0, A, 4, 0, 0, 0) == INVALID
    assert run(B.FORK, A, 0, 0, 0, 1, 0, 0, 0) == INVALID            # no sources
    assert run(B.COMPACT, A, 0, 0, 0, 1, 0, 0, 0) == INVALID and run(B.COMPACT, A, A, 0, 0, -1, 0, 0, 0) == INVALID
    assert run(B.RESERVE, 0, 0, 0, 0, 0, 0, 0, 0) == INVALID


def test_every_declared_symbol_is_exported_and_bound():
    lib = B.lib()
    names = B.declared_functions(_build.INCLUDE + "/kvcache.h")
    assert len(names) == 10
    for name in names:
        assert hasattr(lib, name), name
        assert getattr(lib, name).argtypes is not None, name


@pytest.mark.parametrize("kw,code", [
    (dict(layers=0), INVALID), (dict(Hkv=0), INVALID), (dict(pages=0), INVALID), (dict(seqs=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(code=2), INVALID), (dict(d=0), INVALID), (dict(d=60), UNSUPPORTED),
    (dict(d=136), UNSUPPORTED), (dict(page=16), UNSUPPORTED), (dict(page=96), UNSUPPORTED),
    (dict(max_pages=1 << 25), UNSUPPORTED), (dict(pages=(1 << 24) + 1), UNSUPPORTED), (dict(Hkv=4097), UNSUPPORTED)])
def test_shapes_are_refused(kw, code):
    assert calls(shape(**kw), buffers()) == [code] * 6


def test_buffers_and_counts_are_refused():
    for name, _ in B.kvcache_buffers._fields_:
        assert calls(shape(), buffers(**{name: None})) == [INVALID] * 6
        assert calls(shape(), buffers(**{name: A + 8})) == [INVALID] * 6
    assert calls(shape(), buffers(), n=5) == [INVALID] * 6        # more entries than sequences
    assert calls(shape(), buffers(), n=-1) == [INVALID] * 6
    assert calls(shape(), buffers(), status=None) == [INVALID] * 6
    got = calls(shape(), buffers(), layer=2)
    assert got[1] == got[2] == INVALID
    got = calls(shape(), buffers(), wsb=64)
    assert [got[0], got[3], got[4]] == [WORKSPACE] * 3
    got = calls(shape(), buffers(), ws=None)
    assert [got[0], got[3], got[4]] == [WORKSPACE] * 3


def test_calls_without_entries_do_nothing():
    got = calls(shape(), buffers(), n=0)
    assert got == [0] * 6


def test_attention_and_window_arguments():
    L, s, b = B.lib(), shape(), buffers()
    call = lambda q=A, Hq=4, T=1, w=0, k=0, out=A + (1 << 20): L.kvcache_attention(
        ctypes.byref(s), ctypes.byref(b), 0, None, 2, q, Hq, T, w, k, out, A, 1 << 30, A, None)
    assert [call(q=None), call(out=None), call(q=A + 2), call(Hq=3), call(Hq=0), call(T=0), call(w=-1), call(k=-1),
            call(out=A)] == [INVALID] * 9
    assert call(T=1 << 24) == UNSUPPORTED
    win = lambda B_=1, Hq=4, Hkv=2, d=64, n=100, q=A, k=A, v=A, w=5, sk=0, out=A + (1 << 24), st=A: \
        L.kvcache_window_attention(B_, Hq, Hkv, d, n, q, k, v, None, w, sk, out, st, None)
    assert [win(B_=0), win(Hq=3), win(n=0), win(w=-1), win(sk=-1), win(q=None), win(k=A + 8), win(out=A), win(st=None)
            ] == [INVALID] * 9
    assert [win(d=60), win(d=136), win(B_=70000)] == [UNSUPPORTED] * 3


# ------------------------------------------------------------------ the reference itself
def test_reference_rounds_like_the_formats():
    torch = pytest.importorskip("torch")
    x = torch.linspace(-460, 460, 20001, dtype=torch.float64)
    x = torch.cat((x[x.abs() <= 448], torch.exp2(torch.linspace(-12, 8, 5001, dtype=torch.float64))))
    want = x.float().to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(R.to_e4m3(x.float().double().numpy()), want)
    for amax, s in ((448.0, 1.0), (449.0, 2.0), (3.5, 2.0 ** -7), (0.0, 2.0 ** -120), (1e-40, 2.0 ** -120)):
        assert R.page_scale(amax, "e4m3") == s


def test_reference_program():
    r = R.RefCache(3, 1, 8, 6, 32, 4, 1, "int8")
    r.reserve([40, 1, 0])
    assert r.table == [[0, 1], [2], []] and r.refs == [1, 1, 1, 0, 0, 0]
    r.fork([0], [2])
    assert r.table[2] == [0, 3] and r.refs == [2, 1, 1, 1, 0, 0]
    r.compact([[[[0, 39]]]], [2], [0])
    assert r.table[0] == [4] and r.refs == [1, 0, 1, 1, 1, 0] and r.length == [2, 1, 40]
    r.free([2])
    r.reserve([70, 0, 0])
    assert r.table[0] == [4, 0, 1] and r.flags == 0
    r.reserve([0, 0, 97])
    assert r.flags == R.FLAG["NO_PAGES"] and r.length[2] == 0
