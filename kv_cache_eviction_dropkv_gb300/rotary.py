"""Norms and positions of queries and keys.

The kernels are in libdropkv.so (include/kvcache_step.h); this module makes
the table of frequencies, owns it and checks arguments.
"""
from __future__ import annotations

import math
from typing import Optional

import torch

from . import _binding as B

LAYOUTS = {"half": 0, "interleaved": 1}
_SCALINGS = {"linear": {"factor"}, "ntk": {"factor"}, "yarn": {"factor", "original", "fast", "slow", "amplitude"},
             "bands": {"factor", "original", "low", "high"}}


def frequencies(dims: int, base: float = 10000.0, scaling: Optional[dict] = None):
    """Radians per position of the dims / 2 pairs, base^(-2 i / dims) changed
    by `scaling` (Rotary's), and the amplitude: ([float], float)."""
    if not (math.isfinite(base) and base > 0):
        raise ValueError("base must be positive")
    how = {k: v for k, v in (scaling or {}).items() if v is not None}
    kind = how.pop("kind", None)
    if scaling:
        if kind not in _SCALINGS or not {"factor"} <= set(how) <= _SCALINGS[kind]:
            raise ValueError("scaling: kind is one of %s, with %s" % (sorted(_SCALINGS), {k: sorted(v) for k, v in
                                                                                          _SCALINGS.items()}))
        if any(not (math.isfinite(v) and v > 0) for v in how.values()):
            raise ValueError("scaling: positive numbers are wanted")
    factor, amplitude = float(how.get("factor", 1.0)), 1.0
    if kind == "ntk" and dims > 2:
        base = base * factor ** (dims / (dims - 2))
    freq = [base ** (-2.0 * i / dims) for i in range(dims // 2)]
    if kind in ("yarn", "bands") and "original" not in how:
        raise ValueError("scaling: %s needs the original context length" % kind)
    if kind == "linear":
        freq = [f / factor for f in freq]
    elif kind == "bands":
        low, high = float(how.get("low", 1.0)), float(how.get("high", 4.0))
        if high <= low:
            raise ValueError("scaling: high must be above low")
        for i, f in enumerate(freq):
            keep = min(1.0, max(0.0, (how["original"] * f / (2 * math.pi) - low) / (high - low)))
            freq[i] = f / factor * (1 - keep) + f * keep
    elif kind == "yarn":
        if base <= 1:
            raise ValueError("scaling: yarn needs a base above 1")
        fast, slow = float(how.get("fast", 32.0)), float(how.get("slow", 1.0))
        if fast < slow:
            raise ValueError("scaling: fast must not be below slow")
        edge = lambda turns: dims * math.log(how["original"] / (2 * math.pi * turns)) / (2 * math.log(base))
        lo, hi = max(0, math.floor(edge(fast))), min(dims - 1, math.ceil(edge(slow)))
        for i, f in enumerate(freq):
            keep = 1.0 - min(1.0, max(0.0, (i - lo) / max(0.001, hi - lo)))
            freq[i] = f / factor * (1 - keep) + f * keep
        amplitude = how.get("amplitude")
        amplitude = 0.1 * math.log(max(1.0, factor)) + 1.0 if amplitude is None else float(amplitude)
    return freq, amplitude


class Rotary:
    """What a layer does to its queries and keys before they meet: an RMS norm
    of each head (where there are weights), then the rotation of its first
    `dims` channels by their position.  A plan: made once, used by apply(),
    and by PagedCache.store_rotated() for tokens that go into the cache."""

    def __init__(self, d: int, dims: Optional[int] = None, base: float = 10000.0, layout: str = "half",
                 scaling: Optional[dict] = None, q_norm=None, k_norm=None, eps: float = 1e-6, device=None):
        """d: channels of a head; dims: how many of them turn (default: all; 0:
        norm only); layout: "half" (channels i and i + dims / 2 are a pair) or
        "interleaved" (2 i and 2 i + 1); q_norm, k_norm: weights [d], or None.
        scaling, for contexts longer than those of the training: None, or one
        of dict(kind="linear", factor=) all frequencies / factor; "ntk": base *
        factor^(dims / (dims - 2)); "yarn" (original=, fast=32, slow=1): pairs
        that turn more than `fast` times over the original context stay, those
        below `slow` are divided, a ramp over the pairs between, and the
        rotated channels are multiplied by amplitude (default 0.1 ln(factor) +
        1, or 1 for a factor below 1); "bands" (original=, low=1, high=4): the
        same with a ramp over the turns and no amplitude."""
        self.d, self.dims, self.eps = int(d), int(d if dims is None else dims), float(eps)
        if not 8 <= self.d <= 128 or self.d % 8 or not 0 <= self.dims <= self.d or self.dims % 8:
            raise ValueError("d is a multiple of 8 up to 128, dims one up to d")
        if layout not in LAYOUTS:
            raise ValueError("layout must be one of %s" % sorted(LAYOUTS))
        if not (math.isfinite(self.eps) and self.eps > 0):
            raise ValueError("eps must be positive")
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        if self.device.type != "cuda":
            raise ValueError("the plan lives on a CUDA device")
        freq, self.amplitude = frequencies(self.dims, base, scaling)
        # turns per position as 64-bit fractions: a position times one, modulo
        # 2^64, is the angle
        turns = [round(f / (2 * math.pi) * 2.0 ** 64) % (1 << 64) for f in freq]
        turns = [t - (1 << 64) if t >= 1 << 63 else t for t in turns]
        with torch.cuda.device(self.device):
            self.device = torch.device("cuda", torch.cuda.current_device())
            self.turns = torch.tensor(turns, dtype=torch.int64, device=self.device)
            self.q_norm, self.k_norm = (self._weight(n, w) for n, w in (("q_norm", q_norm), ("k_norm", k_norm)))
            self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._index = self.device.index
        address = lambda t: None if t is None or t.numel() == 0 else t.data_ptr()
        self._record = B.kvcache_rotary(address(self.turns), address(self.q_norm), address(self.k_norm), self.d,
                                        self.dims, LAYOUTS[layout], self.eps, self.amplitude)
        self.address, self._status = B.address_of(self._record), self.status.data_ptr()

    def _weight(self, name, w):
        if w is None:
            return None
        if w.shape != (self.d,):
            raise ValueError("%s: expected [%d] weights" % (name, self.d))
        return w.detach().to(self.device, torch.float32).clone().contiguous()

    def apply(self, q, k, q_out, k_out, positions=None, lengths=None, stream=None):
        """q [B, Hq, n, d] and k [B, Hkv, n, d] bf16, of any strides with adjacent
        channels (views of a packed projection, for instance; rows 16-byte
        aligned), into contiguous q_out and k_out; q or k may be None or have no
        heads, and q_out may be q itself where that is contiguous.  positions:
        int32 [B], row t of sequence b stands at positions[b] + t; int32 [B, n],
        one for each row; None: row t at t.  Rows from lengths[b] (int32 [B]) on
        are left as they were.  Problems found on the device are reported by
        check()."""
        if q is not None and q.shape[1] == 0:
            q = None
        if k is not None and k.shape[1] == 0:
            k = None
        if q is None and k is None:
            return
        i, d = self._index, self.d
        n_seq, _, n, _ = (k if q is None else q).shape
        Hq = Hkv = 1
        of_q = of_k = B.NO_ROWS
        to_q = to_k = 0
        if q is not None:
            Hq = q.shape[1]
            want = (n_seq, Hq, n, d)
            of_q = B.rows_of("q", q, want, i)
            to_q = B.tensor_address("q_out", q_out, B.bf16, want, i)
        if k is not None:
            Hkv = k.shape[1]
            want = (n_seq, Hkv, n, d)
            of_k = B.rows_of("k", k, want, i)
            to_k = B.tensor_address("k_out", k_out, B.bf16, want, i)
        at, kind = B.positions_of(positions, n_seq, n, i)
        to = 0 if lengths is None else B.tensor_address("lengths", lengths, B.int32, (n_seq,), i)
        if not (n_seq and n):
            return
        if B.current_device() != i:
            with torch.cuda.device(self.device):
                return self.apply(q, k, q_out, k_out, positions, lengths, stream)
        code = B.lib().kvcache_rotate(B.rotate_call.pack(
            self.address, *of_q, *of_k, to_q, to_k, at, to, self._status,
            B.current_raw_stream(i) if stream is None else B.raw_stream(stream), n_seq, Hq, Hkv, n, kind))
        if code != 0:
            raise B.DropKVError(code, "kvcache_rotate")

    def check(self, stream=None):
        """Sync and raise if the device status word reports an error."""
        with torch.cuda.device(self.device):
            code, flags = B.kvcache_read_status(self.status, stream)
        if code != 0:
            raise B.DropKVError(code, "device status 0x%x" % flags)
        return flags

    def reset_status(self):
        self.status.zero_()
