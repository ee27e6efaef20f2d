"""ctypes binding of libdropkv.so (include/dropkv.h, include/kvcache.h and
include/kvcache_step.h), same names as the C ABI.

Argument marshalling only: tensors are passed as device pointers and the
current torch stream as the CUDA stream; every step runs in the library.  If
the library has not been built, the first call raises; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct
import threading

import torch

from . import _build

STATUS_NAMES = {0: "OK", 1: "INVALID_ARG", 2: "WORKSPACE", 3: "SINGULAR", 4: "NONFINITE", 5: "CUDA",
                6: "UNSUPPORTED", 7: "DEVICE_ARG", 8: "TIMEOUT"}
FLAG_SINGULAR, FLAG_NONFINITE, FLAG_BAD_LENGTH, FLAG_BAD_K, FLAG_OVERFLOW, FLAG_TIMEOUT = 1, 2, 4, 8, 16, 32
FLAG_NO_PAGES, FLAG_BAD_SEQ, FLAG_BAD_PAGE = 0x1000, 0x2000, 0x4000


class DropKVError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__("%s failed: DROPKV_ERR_%s (%d)" % (where, STATUS_NAMES.get(code, "?"), code))
        self.code = code


class dropkv_shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("d", ctypes.c_int32), ("n_max", ctypes.c_int32), ("w", ctypes.c_int32)]

    def astuple(self):
        return (self.B, self.Hq, self.Hkv, self.d, self.n_max, self.w)


CACHE_CODES = {"e4m3": 0, "int8": 1}


class kvcache_shape(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int32) for name in ("layers", "Hkv", "d", "page", "pages", "seqs", "max_pages", "code")]


class kvcache_buffers(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in ("k", "v", "k_scale", "v_scale", "refs", "table", "count", "length")]


class kvcache_rotary(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p),
                ("d", ctypes.c_int32), ("dims", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("eps", ctypes.c_float), ("amplitude", ctypes.c_float)]


STEP_CALLS = ("kvcache_rotate", "kvcache_rotate_store", "kvcache_read", "kvcache_shared_attention")

_lock = threading.Lock()
_lib = None
_active = None          # a library loaded by use_library(), else None


def library_path() -> str:
    return _build.LIB_PATH


def _load(path):
    if not os.path.exists(path):
        raise RuntimeError("%s is not built; run __graft_entry__.build()" % path)
    L = ctypes.CDLL(path)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    SH = ctypes.POINTER(dropkv_shape)
    L.dropkv_workspace_size.argtypes = [SH]
    L.dropkv_workspace_size.restype = SZ
    L.dropkv_score.argtypes = [SH, P, P, P, P, I32, I32, P, P, P, SZ, P, P]
    L.dropkv_score.restype = ctypes.c_int
    L.dropkv_score_timed.argtypes = [SH, I32, P, P, P, P, I32, I32, P, P, P, SZ, P, P, P]
    L.dropkv_score_timed.restype = ctypes.c_int
    L.dropkv_score_noalloc.argtypes = [SH, P, P, P, P, I32, I32, P, P, P, P]
    L.dropkv_score_noalloc.restype = ctypes.c_int
    L.dropkv_select.argtypes = [SH, P, P, P, I32, P, P, P, SZ, P, P]
    L.dropkv_select.restype = ctypes.c_int
    L.dropkv_compact.argtypes = [SH, P, P, P, P, I32, P, P, P, P]
    L.dropkv_compact.restype = ctypes.c_int
    L.dropkv_evict.argtypes = [SH, P, P, P, P, P, I32, I32, P, P, P, P, I32, P, P, P, SZ, P, P]
    L.dropkv_evict.restype = ctypes.c_int
    L.dropkv_evict_ex.argtypes = [SH, I32, P, P, P, P, P, I32, I32, P, P, P, P, I32, P, P, P, SZ, P, P]
    L.dropkv_evict_ex.restype = ctypes.c_int
    L.dropkv_evict_prefill.argtypes = [SH, I32, P, P, P, P, P, I32, I32, P, P, P, P, P, I32, P, P, P, SZ, P, P]
    L.dropkv_evict_prefill.restype = ctypes.c_int
    L.dropkv_prefill_attention.argtypes = [SH, P, P, P, P, P, P, SZ, P, P]
    L.dropkv_prefill_attention.restype = ctypes.c_int
    L.dropkv_score_ex.argtypes = [SH, I32, P, P, P, P, I32, I32, P, P, P, SZ, P, P]
    L.dropkv_score_ex.restype = ctypes.c_int
    L.dropkv_select_layer.argtypes = [SH, P, P, P, I32, P, P, P, SZ, P, P]
    L.dropkv_select_layer.restype = ctypes.c_int
    L.dropkv_compact_heads.argtypes = [SH, P, P, P, P, I32, P, P, P, P]
    L.dropkv_compact_heads.restype = ctypes.c_int
    L.dropkv_read_status.argtypes = [P, P, ctypes.POINTER(ctypes.c_uint32)]
    L.dropkv_read_status.restype = ctypes.c_int
    L.dropkv_version.argtypes = []
    L.dropkv_version.restype = ctypes.c_char_p
    CS, CB = ctypes.POINTER(kvcache_shape), ctypes.POINTER(kvcache_buffers)
    L.kvcache_workspace_size.argtypes = [CS, I32, I32]
    L.kvcache_workspace_size.restype = SZ
    for name, args in (
            ("kvcache_reserve", [CS, CB, P, I32, P, P, SZ, P, P]),
            ("kvcache_store", [CS, CB, I32, P, I32, P, P, I32, P, P, P]),
            ("kvcache_attention", [CS, CB, I32, P, I32, P, I32, I32, I32, I32, P, P, SZ, P, P]),
            ("kvcache_fork", [CS, CB, P, P, I32, I32, P, SZ, P, P]),
            ("kvcache_compact", [CS, CB, P, I32, P, I32, P, P, SZ, P, P]),
            ("kvcache_free", [CS, CB, P, I32, P, P]),
            ("kvcache_run", [ctypes.c_char_p]),
            ("kvcache_window_attention", [I32, I32, I32, I32, I32, P, P, P, P, I32, I32, P, P, P]),
            ("kvcache_read_status", [P, P, ctypes.POINTER(ctypes.c_uint32)])):
        getattr(L, name).argtypes = args
        getattr(L, name).restype = ctypes.c_int
    L.kvcache_shared_workspace_size.argtypes = [CS, I32, I32, I32, I32]
    L.kvcache_shared_workspace_size.restype = SZ
    for name in STEP_CALLS:
        getattr(L, name).argtypes = [ctypes.c_char_p]
        getattr(L, name).restype = ctypes.c_int
    for hook in ("dropkv_test_skip_pass2_k", "dropkv_test_skip_prefill_k", "kvcache_test_skip_window_pair",
                 "kvcache_test_skip_shared_load"):
        if hasattr(L, hook):
            getattr(L, hook).argtypes = [I32, I32]
            getattr(L, hook).restype = ctypes.c_int
    return L


def lib():
    """The library the calls go to: libdropkv.so (raises if it was not
    built), or the one a use_library() block selected."""
    global _lib
    if _active is not None:
        return _active
    if _lib is None:
        with _lock:
            if _lib is None:
                _lib = _load(_build.LIB_PATH)
    return _lib


class use_library:
    """Route this module's calls to another build of the library (the test
    build of include/dropkv_test_hooks.h) inside a with-block."""

    _cache = {}

    def __init__(self, path):
        with _lock:
            if path not in self._cache:
                self._cache[path] = _load(path)
        self.L = self._cache[path]

    def __enter__(self):
        global _active
        self.prev, _active = _active, self.L
        return self.L

    def __exit__(self, *exc):
        global _active
        _active = self.prev
        return False


def declared_functions(header: str = None):
    """Names of the functions include/dropkv.h declares."""
    header = header or os.path.join(_build.INCLUDE, "dropkv.h")
    text = open(header).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b((?:dropkv|kvcache)_[a-z0-9_]+)\s*\(", text)))


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch tensor")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("tensors must be contiguous CUDA tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def make_shape(B, Hq, Hkv, d, n_max, w) -> dropkv_shape:
    return dropkv_shape(int(B), int(Hq), int(Hkv), int(d), int(n_max), int(w))


def _check(code, where):
    if code != 0:
        raise DropKVError(code, where)
    return code


def dropkv_workspace_size(shape: dropkv_shape) -> int:
    return int(lib().dropkv_workspace_size(ctypes.byref(shape)))


def dropkv_score(shape, q_window, k, v, lengths, pool_kernel, protect, scores, raw_scores, workspace, status,
                 stream=None):
    code = lib().dropkv_score(ctypes.byref(shape), _ptr(q_window), _ptr(k), _ptr(v), _ptr(lengths),
                              int(pool_kernel), int(protect), _ptr(scores), _ptr(raw_scores), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream))
    return _check(code, "dropkv_score")


def dropkv_score_timed(shape, q_window, k, v, lengths, pool_kernel, protect, scores, raw_scores, workspace,
                       status, events, stream=None, kind="dropkv"):
    """dropkv_score recording 5 torch.cuda.Event objects at its phase boundaries."""
    if len(events) != 5:
        raise ValueError("dropkv_score_timed records 5 events")
    arr = (ctypes.c_void_p * 5)(*[ctypes.c_void_p(e.cuda_event) for e in events])
    code = lib().dropkv_score_timed(ctypes.byref(shape), SCORE_KINDS[kind], _ptr(q_window), _ptr(k), _ptr(v),
                                    _ptr(lengths),
                                    int(pool_kernel), int(protect), _ptr(scores), _ptr(raw_scores),
                                    _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(status),
                                    _stream(stream), arr)
    return _check(code, "dropkv_score_timed")


def dropkv_score_noalloc(shape, q_window, k, v, lengths, pool_kernel, protect, scores, raw_scores, status,
                         stream=None):
    """dropkv_score with the library's fixed scratch array instead of a workspace (allocates nothing)."""
    code = lib().dropkv_score_noalloc(ctypes.byref(shape), _ptr(q_window), _ptr(k), _ptr(v), _ptr(lengths),
                                      int(pool_kernel), int(protect), _ptr(scores), _ptr(raw_scores),
                                      _ptr(status), _stream(stream))
    return _check(code, "dropkv_score_noalloc")


def dropkv_select(shape, scores, lengths, evict_k, protect, kept_idx, kept_len, workspace, status, stream=None):
    code = lib().dropkv_select(ctypes.byref(shape), _ptr(scores), _ptr(lengths), _ptr(evict_k), int(protect),
                               _ptr(kept_idx), _ptr(kept_len), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream))
    return _check(code, "dropkv_select")


def dropkv_compact(shape, k, v, kept_idx, kept_len, out_rows, k_out, v_out, status, stream=None):
    code = lib().dropkv_compact(ctypes.byref(shape), _ptr(k), _ptr(v), _ptr(kept_idx), _ptr(kept_len),
                                int(out_rows), _ptr(k_out), _ptr(v_out), _ptr(status), _stream(stream))
    return _check(code, "dropkv_compact")


def dropkv_evict(shape, q_window, k, v, lengths, evict_k, pool_kernel, protect, scores, raw_scores, kept_idx,
                 kept_len, out_rows, k_out, v_out, workspace, status, stream=None):
    code = lib().dropkv_evict(ctypes.byref(shape), _ptr(q_window), _ptr(k), _ptr(v), _ptr(lengths), _ptr(evict_k),
                              int(pool_kernel), int(protect), _ptr(scores), _ptr(raw_scores), _ptr(kept_idx),
                              _ptr(kept_len), int(out_rows), _ptr(k_out), _ptr(v_out), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream))
    return _check(code, "dropkv_evict")


SCORE_KINDS = {"dropkv": 0, "snapkv": 1}


def dropkv_score_ex(shape, kind, q_window, k, v, lengths, pool_kernel, protect, scores, raw_scores, workspace,
                    status, stream=None):
    code = lib().dropkv_score_ex(ctypes.byref(shape), SCORE_KINDS[kind], _ptr(q_window), _ptr(k), _ptr(v),
                                 _ptr(lengths), int(pool_kernel), int(protect), _ptr(scores), _ptr(raw_scores),
                                 _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(status),
                                 _stream(stream))
    return _check(code, "dropkv_score_ex")


def dropkv_evict_ex(shape, kind, q_window, k, v, lengths, evict_k, pool_kernel, protect, scores, raw_scores,
                    kept_idx, kept_len, out_rows, k_out, v_out, workspace, status, stream=None):
    code = lib().dropkv_evict_ex(ctypes.byref(shape), SCORE_KINDS[kind], _ptr(q_window), _ptr(k), _ptr(v),
                                 _ptr(lengths), _ptr(evict_k), int(pool_kernel), int(protect), _ptr(scores),
                                 _ptr(raw_scores), _ptr(kept_idx), _ptr(kept_len), int(out_rows), _ptr(k_out),
                                 _ptr(v_out), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _ptr(status), _stream(stream))
    return _check(code, "dropkv_evict_ex")


def dropkv_evict_prefill(shape, kind, q, k, v, lengths, evict_k, pool_kernel, protect, attn_out, scores, raw_scores,
                         kept_idx, kept_len, out_rows, k_out, v_out, workspace, status, stream=None):
    _check(lib().dropkv_evict_prefill(ctypes.byref(shape), SCORE_KINDS[kind], _ptr(q), _ptr(k), _ptr(v), _ptr(lengths),
                                      _ptr(evict_k), int(pool_kernel), int(protect), _ptr(attn_out), _ptr(scores),
                                      _ptr(raw_scores), _ptr(kept_idx), _ptr(kept_len), int(out_rows), _ptr(k_out),
                                      _ptr(v_out), _ptr(workspace), workspace.numel(), _ptr(status),
                                      _stream(stream)), "dropkv_evict_prefill")


def dropkv_prefill_attention(shape, q, k, v, lengths, attn_out, workspace, status, stream=None):
    _check(lib().dropkv_prefill_attention(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(lengths),
                                          _ptr(attn_out), _ptr(workspace), workspace.numel(), _ptr(status),
                                          _stream(stream)), "dropkv_prefill_attention")


def dropkv_select_layer(shape, scores, lengths, evict_total, protect, kept_idx, kept_len, workspace, status,
                        stream=None):
    code = lib().dropkv_select_layer(ctypes.byref(shape), _ptr(scores), _ptr(lengths), _ptr(evict_total),
                                     int(protect), _ptr(kept_idx), _ptr(kept_len), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream))
    return _check(code, "dropkv_select_layer")


def dropkv_compact_heads(shape, k, v, kept_idx, kept_len, out_rows, k_out, v_out, status, stream=None):
    code = lib().dropkv_compact_heads(ctypes.byref(shape), _ptr(k), _ptr(v), _ptr(kept_idx), _ptr(kept_len),
                                      int(out_rows), _ptr(k_out), _ptr(v_out), _ptr(status), _stream(stream))
    return _check(code, "dropkv_compact_heads")


def dropkv_read_status(status, stream=None):
    """Sync the stream and return (status code, raw flag word)."""
    flags = ctypes.c_uint32(0)
    code = lib().dropkv_read_status(_ptr(status), _stream(stream), ctypes.byref(flags))
    return int(code), int(flags.value)


def dropkv_version() -> str:
    return lib().dropkv_version().decode()


# ------------------------------------------------------------------ include/kvcache.h
# Small calls (one new token) cost a few microseconds, so these go with raw
# addresses and streams, and as few layers as can be: PagedCache packs a
# kvcache_call record and makes its calls through lib() directly (an argument
# that ctypes converts costs 0.1 us, the whole record 0.2).  Plain lookups of
# the current stream's handle and the current device: building a Stream object
# would add two microseconds.
kvcache_call = struct.Struct("@PPPNPPPPPPP7i0P")   # the fields of the record, in order
RESERVE, STORE, ATTENTION, FORK, COMPACT, FREE = range(6)
RESERVE_GRANTED = 16 + RESERVE
CACHE_CALLS = tuple("kvcache_" + name for name in ("reserve", "store", "attention", "fork", "compact", "free"))
current_raw_stream, current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def raw_stream(stream) -> int:
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def kvcache_workspace_size(shape, Hq, T) -> int:
    return int(lib().kvcache_workspace_size(ctypes.byref(shape), int(Hq), int(T)))


def kvcache_window_attention(device_index, B, Hq, Hkv, d, n_max, q, k, v, lengths, window, sinks, attn_out, status,
                             stream=None):
    """Raw addresses (lengths: or None) on the device of that index."""
    if current_device() != device_index:
        with torch.cuda.device(device_index):
            return kvcache_window_attention(device_index, B, Hq, Hkv, d, n_max, q, k, v, lengths, window, sinks,
                                            attn_out, status, stream)
    _check(lib().kvcache_window_attention(B, Hq, Hkv, d, n_max, q, k, v, lengths, window, sinks, attn_out, status,
                                          current_raw_stream(device_index) if stream is None else raw_stream(stream)),
           "kvcache_window_attention")


def kvcache_read_status(status, stream=None):
    """Sync the stream and return (status code, raw flag word)."""
    flags = ctypes.c_uint32(0)
    code = lib().kvcache_read_status(_ptr(status), _stream(stream), ctypes.byref(flags))
    return int(code), int(flags.value)


# ------------------------------------------------------------------ include/kvcache_step.h
# Its calls take one record each, packed here field by field.
rotate_call = struct.Struct("@P" + "P3q" * 2 + "6P" + "5i0P")
rotate_store_call = struct.Struct("@3P" + "P3q" * 3 + "6P" + "5i0P")
read_call = struct.Struct("@9P3i0P")
shared_attention_call = struct.Struct("@7PN2Pq5i0P")
address_of = ctypes.addressof


def bad_tensor(name, t, dtype, shape, device_index):
    """What a call says of a tensor that it has no use for."""
    return ValueError("%s: expected a contiguous %s %s tensor on device %d, got %s %s on %s"
                      % (name, dtype, list(shape), device_index, t.dtype, list(t.shape), t.device))


def tensor_address(name, t, dtype, shape, device_index):
    """Address of a contiguous tensor of that type and shape on the device of that index."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device_index or not t.is_contiguous():
        raise bad_tensor(name, t, dtype, shape, device_index)
    return t.data_ptr()


bf16, int32 = torch.bfloat16, torch.int32


def rows_of(name, t, shape, device_index):
    """Address and strides of bf16 rows [sequences][heads][rows][d] (kvcache_rows)."""
    if t.dtype is not bf16 or t.shape != shape or t.get_device() != device_index:
        raise ValueError("%s: expected a bf16 %s tensor on device %d, got %s %s on %s"
                         % (name, list(shape), device_index, t.dtype, list(t.shape), t.device))
    a = t.data_ptr()
    s0, s1, s2, s3 = strides = t.stride()
    if (s3 != 1 or a & 15 or (s0 | s1 | s2) & 7) and (
            s3 != 1 or a & 15 or any(s & 7 and n > 1 for s, n in zip(strides[:3], shape))):
        raise ValueError("%s: rows of adjacent channels on 16-byte boundaries are wanted, got strides %s"
                         % (name, list(strides)))
    return a, s0, s1, s2


NO_ROWS = (0, 0, 0, 0)


def positions_of(positions, n, rows, device_index):
    """Address and kind of a call's positions (None, int32 [n] or [n, rows])."""
    if positions is None:
        return 0, 0
    each = positions.dim() == 2
    return tensor_address("positions", positions, int32, (n, rows) if each else (n,), device_index), int(each)


def kvcache_shared_workspace_size(shape, n, Hq, T, G) -> int:
    return int(lib().kvcache_shared_workspace_size(ctypes.byref(shape), int(n), int(Hq), int(T), int(G)))
