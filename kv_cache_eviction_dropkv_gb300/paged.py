"""A paged KV cache in 8 bits: where an eviction's kept rows go, and what
decoding reads.

Every computation runs in libdropkv.so (include/kvcache.h); this module owns
the buffers and checks arguments.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _binding as B

DTYPES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


class PagedCache:
    """Pages of keys and values for up to `seqs` sequences on one device.

    A step of a serving loop is reserve() (make room for the new tokens), then
    per layer store() (their keys and values) and attention() (their queries).
    fork(), copy(), compact() and free() work on whole sequences, all layers at
    once.  Calls run on the current stream of the cache's device (or `stream`)
    in the order they are made; calls on one cache, or on one workspace, that
    would overlap on the GPU are the caller's to order.  Problems found on the
    device (a sequence that does not exist, too few free pages, ...) are
    reported by check().  A store() behind a reserve() that was refused would
    replace the sequence's last tokens: where pages or table entries can run
    out between two check()s, pass what was granted on (reserve(granted=),
    store(counts=)).

    Buffers (device tensors, free to read): k, v [layers, pages, Hkv, page, d]
    codes, k_scale, v_scale [layers, pages, Hkv], refs [pages], table
    [seqs, max_pages], count and length [seqs]."""

    def __init__(self, seqs: int, Hkv: int, d: int, pages: int, page: int = 64, max_pages: Optional[int] = None,
                 layers: int = 1, code: str = "e4m3", Hq: Optional[int] = None, T: int = 1, device=None):
        """pages: pages in the pool; page: tokens per page (32, 64 or 128);
        max_pages: most pages of one sequence (default: all; attention over
        short sequences is faster with a bound near their length); code: "e4m3" or
        "int8"; Hq, T: query heads (default: Hkv) and most query rows per
        sequence of an attention() call (they size the workspace)."""
        if code not in B.CACHE_CODES:
            raise ValueError("code must be one of %s" % sorted(B.CACHE_CODES))
        max_pages = pages if max_pages is None else max_pages
        self.layers, self.Hkv, self.d, self.page, self.pages = int(layers), int(Hkv), int(d), int(page), int(pages)
        self.seqs, self.max_pages, self.code = int(seqs), int(max_pages), code
        self.Hq, self.T = int(Hkv if Hq is None else Hq), int(T)
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        if self.device.type != "cuda":
            raise ValueError("the cache lives on a CUDA device")
        self.shape = B.kvcache_shape(self.layers, self.Hkv, self.d, self.page, self.pages, self.seqs, self.max_pages,
                                     B.CACHE_CODES[code])
        with torch.cuda.device(self.device):
            self.device = torch.device("cuda", torch.cuda.current_device())
            ws = B.kvcache_workspace_size(self.shape, self.Hq, self.T)
            if ws == 0:
                raise B.DropKVError(6, "kvcache_workspace_size")
            dev = self.device
            self.workspace = torch.empty(ws, dtype=torch.uint8, device=dev)
            self.status = torch.zeros(1, dtype=torch.int32, device=dev)
            pool, scales = (self.layers, self.pages, self.Hkv, self.page, self.d), (self.layers, self.pages, self.Hkv)
            self.k = torch.zeros(pool, dtype=DTYPES[code], device=dev)
            self.v = torch.zeros(pool, dtype=DTYPES[code], device=dev)
            self.k_scale = torch.zeros(scales, dtype=torch.float32, device=dev)
            self.v_scale = torch.zeros(scales, dtype=torch.float32, device=dev)
            self.refs = torch.zeros(self.pages, dtype=torch.int32, device=dev)
            self.table = torch.full((self.seqs, self.max_pages), -1, dtype=torch.int32, device=dev)
            self.count = torch.zeros(self.seqs, dtype=torch.int32, device=dev)
            self.length = torch.zeros(self.seqs, dtype=torch.int32, device=dev)
        self._index = self.device.index
        self._buffers = B.kvcache_buffers(*(t.data_ptr() for t in (self.k, self.v, self.k_scale, self.v_scale, self.refs,
                                                                    self.table, self.count, self.length)))
        self._fixed = (ctypes.addressof(self.shape), ctypes.addressof(self._buffers), self.workspace.data_ptr(), ws,
                       self.status.data_ptr())

    # -------------------------------------------------------------- arguments
    def _tensor(self, name, t, dtype, shape):
        """Address of a contiguous device tensor of that type and shape."""
        if t.dtype is not dtype or t.shape != shape or t.get_device() != self._index or not t.is_contiguous():
            raise ValueError("%s: expected a contiguous %s %s tensor on %s, got %s %s on %s"
                             % (name, dtype, list(shape), self.device, t.dtype, list(t.shape), t.device))
        return t.data_ptr()

    def _ints(self, name, t, *shape):
        return self._tensor(name, t, torch.int32, shape)

    def _entries(self, seqs, n):
        """Address of the sequence numbers of a call with n entries (None: 0 .. n - 1)."""
        if n > self.seqs:
            raise ValueError("%d entries, but the cache has %d sequences" % (n, self.seqs))
        return 0 if seqs is None else self._tensor("seqs", seqs, torch.int32, (n,))

    def _layer(self, layer):
        if not 0 <= layer < self.layers:
            raise ValueError("layer %d of a cache with %d" % (layer, self.layers))
        return layer

    def _call(self, op, stream, n, seqs=0, in0=0, in1=0, in2=0, out=0, layer=0, arg0=0, arg1=0, arg2=0, arg3=0):
        """The library's call `op` on the cache, on `stream` (None: the current one of its device)."""
        if n == 0:                                # (an empty tensor has no address)
            return
        if B.current_device() != self._index:
            with torch.cuda.device(self.device):
                return self._call(op, stream, n, seqs, in0, in1, in2, out, layer, arg0, arg1, arg2, arg3)
        code = B.lib().kvcache_run(B.kvcache_call.pack(
            *self._fixed, B.current_raw_stream(self._index) if stream is None else B.raw_stream(stream),
            seqs, in0, in1, in2, out, op, layer, n, arg0, arg1, arg2, arg3))
        if code != 0:
            raise B.DropKVError(code, B.CACHE_CALLS[op & 15])

    # -------------------------------------------------------------- a step
    def reserve(self, extra, seqs=None, stream=None, granted=None):
        """Room for extra[i] more tokens of sequence seqs[i] (int32 [n]); their
        lengths grow.  All or nothing when pages run out.  granted (int32 [n])
        takes extra[i], or 0 where the entry was refused: as store()'s counts
        it keeps a refused step from replacing the tokens before it."""
        n = extra.shape[0]
        to = 0 if granted is None else self._ints("granted", granted, n)
        self._call(B.RESERVE if granted is None else B.RESERVE_GRANTED, stream, n, self._entries(seqs, n),
                   self._ints("extra", extra, n), out=to)

    def store(self, layer, k, v, counts=None, seqs=None, stream=None):
        """Rows 0 .. counts[i] - 1 (default: all) of k, v [n, Hkv, rows, d] bf16
        become the last counts[i] tokens of sequence seqs[i] in `layer`."""
        n, _, rows, _ = k.shape
        want, bf16 = (n, self.Hkv, rows, self.d), torch.bfloat16
        self._call(B.STORE, stream, n if rows else 0, self._entries(seqs, n), self._tensor("k", k, bf16, want),
                   self._tensor("v", v, bf16, want), 0 if counts is None else self._ints("counts", counts, n), 0,
                   self._layer(layer), rows)

    def attention(self, layer, q, out, window: int = 0, sinks: int = 0, seqs=None, stream=None):
        """Attention of the last T tokens of each sequence, q [n, Hq, T, d] bf16,
        into out (same shape): row t stands at position length - T + t and sees
        the tokens up to it; with a window only the last `window` of them and
        the first `sinks` tokens of the sequence."""
        n, Hq, T, _ = q.shape
        if T > self.T or Hq != self.Hq:
            raise ValueError("the workspace is sized for %d query heads and at most %d rows, got %d and %d"
                             % (self.Hq, self.T, Hq, T))
        if T == 0 or n == 0:
            return
        if not (-1 << 31 <= window < 1 << 31 and -1 << 31 <= sinks < 1 << 31):   # (the library refuses negative ones)
            raise ValueError("window and sinks are 32-bit counts")
        want, bf16 = (n, Hq, T, self.d), torch.bfloat16
        self._call(B.ATTENTION, stream, n, self._entries(seqs, n), self._tensor("q", q, bf16, want), 0, 0,
                   self._tensor("out", out, bf16, want), self._layer(layer), Hq, T, window, sinks)

    # -------------------------------------------------------------- whole sequences
    def fork(self, src, dst, stream=None):
        """Empty sequences dst[i] become branches of src[i] (int32 [n]): full
        pages are shared, the partly filled last one is copied."""
        self._branch(src, dst, 1, stream)

    def copy(self, src, dst, stream=None):
        """Empty sequences dst[i] become copies of src[i] that share no page."""
        self._branch(src, dst, 0, stream)

    def _branch(self, src, dst, share, stream):
        n = src.shape[0]
        self._entries(None, n)
        self._call(B.FORK, stream, n, self._ints("src", src, n), self._ints("dst", dst, n), arg0=share)

    def compact(self, kept_idx, kept_len, seqs=None, stream=None):
        """Evict: sequence seqs[i] keeps the kept_len[i] tokens at positions
        kept_idx[layer, i, head, :kept_len[i]] (int32 [layers, n, Hkv, any])."""
        n = kept_len.shape[0]
        stride = kept_idx.shape[-1]
        self._call(B.COMPACT, stream, n, self._entries(seqs, n),
                   self._ints("kept_idx", kept_idx, self.layers, n, self.Hkv, stride),
                   self._ints("kept_len", kept_len, n), arg0=stride)

    def free(self, seqs, stream=None):
        """Release every page of sequences seqs (int32 [n])."""
        n = seqs.shape[0]
        self._call(B.FREE, stream, n, self._entries(seqs, n))

    # -------------------------------------------------------------- status
    def check(self, stream=None):
        """Sync and raise if the device status word reports an error."""
        with torch.cuda.device(self.device):
            code, flags = B.kvcache_read_status(self.status, stream)
        if code != 0:
            raise B.DropKVError(code, "device status 0x%x" % flags)
        return flags

    def reset_status(self):
        self.status.zero_()
