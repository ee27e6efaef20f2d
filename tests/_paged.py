"""Plain reference of the paged 8-bit cache and of the windowed attention: the
state as Python lists and numpy arrays, arithmetic in 64 bits (where the
definition is a 32-bit number, in 32).  Written from the definitions in
include/kvcache.h; shares nothing with the package."""
import math

import numpy as np

SCALE_MIN = 2.0 ** -120
FLAG = dict(NONFINITE=0x2, BAD_LENGTH=0x4, BAD_K=0x8, OVERFLOW=0x10, NO_PAGES=0x1000, BAD_SEQ=0x2000, BAD_PAGE=0x4000)


def page_scale(amax, code):
    if code == "int8":
        return max(float(np.float32(amax) * (np.float32(1) / np.float32(127))), SCALE_MIN)
    if amax == 0:
        return SCALE_MIN
    e = math.ceil(math.log2(amax / 448.0))
    assert amax <= 448.0 * 2.0 ** e and amax > 448.0 * 2.0 ** (e - 1)
    return max(2.0 ** e, SCALE_MIN)


def to_e4m3(x):
    """Nearest e4m3 value (ties to even), saturating; not-a-number stays."""
    x = np.asarray(x, dtype=np.float64)
    a = np.clip(np.where(np.isnan(x), 0.0, np.abs(x)), 0.0, 448.0)
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(a, 1e-300))), -6.0) - 3.0)
    r = np.copysign(np.minimum(np.rint(a / step) * step, 448.0), x)
    return np.where(np.isnan(x), np.nan, r)


def encode(x, scale, code):
    """Code values (as float64) of float64 values x at a scale."""
    if code == "e4m3":
        return to_e4m3(np.asarray(x) / scale)
    with np.errstate(invalid="ignore"):
        q = np.asarray(x, dtype=np.float32) / np.float32(scale)
        return np.where(np.isnan(q), 0.0, np.clip(np.rint(q.astype(np.float64)), -127, 127))


def again(c, was, scale, code):
    """Code values c of scale `was`, rounded again at `scale`."""
    if code == "e4m3":
        return to_e4m3(np.asarray(c) * (was / scale))
    q = np.asarray(c, dtype=np.float32) * np.float32(was) / np.float32(scale)
    return np.clip(np.rint(q.astype(np.float64)), -127, 127)


class RefCache:
    def __init__(self, seqs, Hkv, d, pages, page, max_pages, layers, code):
        self.S, self.H, self.d, self.P, self.page, self.M, self.L, self.code = seqs, Hkv, d, pages, page, max_pages, layers, code
        self.k = np.zeros((layers, pages, Hkv, page, d))
        self.v = np.zeros_like(self.k)
        self.ks = np.zeros((layers, pages, Hkv))
        self.vs = np.zeros_like(self.ks)
        self.refs = [0] * pages
        self.table = [[] for _ in range(seqs)]
        self.length = [0] * seqs
        self.flags = 0

    def _pages(self, tokens):
        return -(-tokens // self.page)

    def _take(self, wanted):
        """The lowest free pages, or None."""
        free = [p for p in range(self.P) if self.refs[p] == 0]
        if len(free) < wanted:
            self.flags |= FLAG["NO_PAGES"]
            return None
        return free[:wanted]

    def reserve(self, extra, seqs=None):
        seqs = list(range(len(extra))) if seqs is None else seqs
        todo, seen = [], set()
        for s, e in zip(seqs, extra):
            if not 0 <= s < self.S or s in seen:
                self.flags |= FLAG["BAD_SEQ"]
                continue
            seen.add(s)
            if e < 0:
                self.flags |= FLAG["BAD_LENGTH"]
            elif self._pages(self.length[s] + e) > self.M:
                self.flags |= FLAG["OVERFLOW"]
            else:
                todo.append((s, e, self._pages(self.length[s] + e) - len(self.table[s])))
        taken = self._take(sum(t[2] for t in todo))
        if taken is None:
            return
        for s, e, need in todo:
            mine, taken = taken[:need], taken[need:]
            for p in mine:
                self.refs[p] = 1
            self.table[s] += mine
            self.length[s] += e

    def store(self, layer, k, v, counts=None, seqs=None):
        n, _, rows, _ = k.shape
        seqs = list(range(n)) if seqs is None else seqs
        seen = set()
        for i, s in enumerate(seqs):
            if not 0 <= s < self.S or s in seen:
                self.flags |= FLAG["BAD_SEQ"]
                continue
            seen.add(s)
            cnt = rows if counts is None else counts[i]
            if cnt < 0 or cnt > rows or cnt > self.length[s]:
                self.flags |= FLAG["BAD_LENGTH"]
                continue
            start = self.length[s] - cnt
            for col in range(start // self.page, self._pages(self.length[s]) if cnt else 0):
                pg = self.table[s][col]
                if self.refs[pg] != 1:
                    self.flags |= FLAG["BAD_PAGE"]
                    continue
                base = col * self.page
                a, z = max(start, base), min(self.length[s], base + self.page)
                for src, codes, scales in ((k, self.k, self.ks), (v, self.v, self.vs)):
                    for h in range(self.H):
                        x = src[i, h, a - start:z - start].astype(np.float64)
                        ok = np.isfinite(x)
                        if not ok.all():
                            self.flags |= FLAG["NONFINITE"]
                        sc = page_scale(float(np.abs(x[ok]).max()) if ok.any() else 0.0, self.code)
                        if a > base:
                            was = scales[layer, pg, h]
                            sc = max(sc, was)
                            old = codes[layer, pg, h, :a - base]
                            if sc > was:
                                codes[layer, pg, h, :a - base] = again(old, was, sc, self.code)
                        codes[layer, pg, h, a - base:z - base] = encode(x, sc, self.code)
                        scales[layer, pg, h] = sc

    def _copy_page(self, a, b):
        for x in (self.k, self.v, self.ks, self.vs):
            x[:, b] = x[:, a]

    def fork(self, src, dst, share=True):
        todo, seen = [], set()
        for s, t in zip(src, dst):
            if not 0 <= s < self.S or not 0 <= t < self.S or t in seen or t in src or self.length[t]:
                self.flags |= FLAG["BAD_SEQ"]
                seen.add(t)
                continue
            seen.add(t)
            both = self.length[s] // self.page if share else 0
            todo.append((s, t, both, len(self.table[s]) - both))
        taken = self._take(sum(x[3] for x in todo))
        if taken is None:
            return
        for s, t, both, need in todo:
            mine, taken = taken[:need], taken[need:]
            for p in self.table[s][:both]:
                self.refs[p] += 1
            for a, b in zip(self.table[s][both:], mine):
                self.refs[b] = 1
                self._copy_page(a, b)
            self.table[t] = self.table[s][:both] + mine
            self.length[t] = self.length[s]

    def compact(self, kept_idx, kept_len, seqs=None):
        seqs = list(range(len(kept_len))) if seqs is None else seqs
        todo, seen = [], set()
        for i, s in enumerate(seqs):
            if not 0 <= s < self.S or s in seen:
                self.flags |= FLAG["BAD_SEQ"]
                continue
            seen.add(s)
            if not 0 <= kept_len[i] <= self.length[s]:
                self.flags |= FLAG["BAD_K"]
                continue
            todo.append((i, s, self._pages(kept_len[i])))
        taken = self._take(sum(x[2] for x in todo))
        if taken is None:
            return
        drop = []
        for i, s, need in todo:
            mine, taken = taken[:need], taken[need:]
            for c, to in enumerate(mine):
                self.refs[to] = 1
                for layer in range(self.L):
                    for h in range(self.H):
                        idx = kept_idx[layer][i][h][c * self.page:min(kept_len[i], (c + 1) * self.page)]
                        frm = [(self.table[s][j // self.page], j % self.page) for j in idx]
                        for codes, scales in ((self.k, self.ks), (self.v, self.vs)):
                            top = max([SCALE_MIN] + [scales[layer, p, h] for p, _ in frm])
                            for r, (p, slot) in enumerate(frm):
                                was = scales[layer, p, h]
                                x = codes[layer, p, h, slot]
                                codes[layer, to, h, r] = x if was == top else again(x, was, top, self.code)
                            scales[layer, to, h] = top
            drop.append((s, mine, kept_len[i]))
        for s, mine, m in drop:
            for p in self.table[s]:
                self.refs[p] -= 1
            self.table[s], self.length[s] = mine, m

    def free(self, seqs):
        for s in seqs:
            if not 0 <= s < self.S:
                self.flags |= FLAG["BAD_SEQ"]
                continue
            for p in self.table[s]:
                self.refs[p] -= 1
            self.table[s], self.length[s] = [], 0

    def values(self, layer, s, h):
        """(K, V) [length][d] of one sequence and head."""
        out = []
        for codes, scales in ((self.k, self.ks), (self.v, self.vs)):
            rows = [codes[layer, p, h] * scales[layer, p, h] for p in self.table[s]]
            out.append(np.concatenate(rows)[:self.length[s]] if rows else np.zeros((0, self.d)))
        return out

    def attention(self, layer, q, window=0, sinks=0, seqs=None):
        """Output [n][Hq][T][d] and, per element row, the largest |v| seen [n][Hq][T]."""
        n, Hq, T, d = q.shape
        seqs = list(range(n)) if seqs is None else seqs
        out, vmax = np.zeros(q.shape), np.zeros(q.shape[:3])
        for i, s in enumerate(seqs):
            for h in range(self.H):
                k, v = self.values(layer, s, h)
                for t in range(T):
                    p = self.length[s] - T + t
                    seen = visible(p, len(k), window, sinks)
                    if not seen.any():
                        continue
                    for hq in range(h * Hq // self.H, (h + 1) * Hq // self.H):
                        out[i, hq, t] = softmax(q[i, hq, t].astype(np.float64) @ k[seen].T / math.sqrt(d)) @ v[seen]
                        vmax[i, hq, t] = np.abs(v[seen]).max()
        return out, vmax


def visible(p, n, window, sinks):
    j = np.arange(n)
    seen = j <= p
    if window:
        seen &= (j > p - window) | (j < sinks)
    return seen


def softmax(x):
    e = np.exp(x - x.max())
    return e / e.sum()


def window_attention(q, k, v, lengths, window, sinks):
    """Output [B][Hq][n][d] (rows >= length zero) and the largest |v| a row sees."""
    B, Hq, n, d = q.shape
    H = k.shape[1]
    out, vmax = np.zeros(q.shape), np.zeros(q.shape[:3])
    for b in range(B):
        L = int(lengths[b])
        i = np.arange(L)[:, None]
        j = np.arange(L)
        seen = (j <= i) & ((j > i - window) | (j < sinks) if window else True)
        for hq in range(Hq):
            h = hq // (Hq // H)
            if L == 0:
                continue
            x = q[b, hq, :L].astype(np.float64) @ k[b, h, :L].astype(np.float64).T / math.sqrt(d)
            x = np.where(seen, x, -np.inf)
            e = np.exp(x - x.max(1, keepdims=True))
            out[b, hq, :L] = e / e.sum(1, keepdims=True) @ v[b, h, :L].astype(np.float64)
            top = np.abs(v[b, h, :L].astype(np.float64)).max(1)
            vmax[b, hq, :L] = np.where(seen, top, 0.0).max(1)
    return out, vmax
