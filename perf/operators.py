"""Workloads of the paged 8-bit KV cache and of the windowed prompt attention.

Each case is one call (or one short run of calls) a serving program makes
around an eviction: it stores the kept keys and values in 8 bits, attends over
them token by token, forks, copies and compacts sequences, and runs the prompt
itself with a sliding window.  `own` selects the package's kernels; otherwise
the same pass is computed in its plain form, elementary torch operations in 32
bits rounded once at the end.  `exact` computes the outputs from the
definitions in 64 bits.

The cache: pages of `page` tokens, codes [layers][pages][Hkv][page][d] in e4m3
or int8, one scale per page and KV head for K and one for V (value = code *
scale); a table of page numbers per sequence; a reference count per page (0 =
free, the lowest free page is taken first).
"""
import math

import torch

own = False

SCALE_MIN = 2.0 ** -120      # smallest scale of a page
QMAX_INT8 = 127.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the first tokens of a chat: one short sequence, one new token; latency
        dict(name="attention_first_tokens", op="attention", code="e4m3", n=1, Hq=32, Hkv=8, d=128, page=64, T=1,
             lo=100, hi=100, window=0, sinks=0),
        # one long document in the headline layer's shape, one new token
        dict(name="attention_long_e4m3", op="attention", code="e4m3", n=1, Hq=32, Hkv=8, d=128, page=64, T=1,
             lo=131072, hi=131072, window=0, sinks=0),
        # the ragged batch of the 28/4-head layer, int8 codes
        dict(name="attention_ragged_int8", op="attention", code="int8", n=4, Hq=28, Hkv=4, d=128, page=128, T=1,
             lo=32768, hi=65535, window=0, sinks=0),
        # a busy server: 48 sequences, four drafted tokens each, sliding window with first tokens kept, MHA d = 96
        dict(name="attention_window_draft4", op="attention", code="e4m3", n=48, Hq=32, Hkv=32, d=96, page=32, T=4,
             lo=3, hi=8191, window=2000, sinks=4),
        # the kept rows of four evicted prompts move into the cache
        dict(name="store_prompts_e4m3", op="store", code="e4m3", n=4, Hkv=8, d=128, page=64, lo=9001, hi=16384,
             old=0, rows=16384),
        # one decode step of 64 sequences: a token each behind partly filled pages
        dict(name="store_step_int8", op="store", code="int8", n=64, Hkv=8, d=128, page=64, lo=1, hi=4095, old=1,
             rows=1),
        # a prompt of 32K tokens with a 4K window
        dict(name="window_prompt_32k", op="window", B=1, Hq=32, Hkv=8, d=128, n=32768, lo=32768, window=4096, sinks=4),
        # a padded batch of short prompts, MHA d = 96, an odd window
        dict(name="window_batch_ragged", op="window", B=4, Hq=32, Hkv=32, d=96, n=2051, lo=1, window=333, sinks=7),
        # parallel samples: 8 prompts forked seven times each, whole pages shared
        dict(name="fork_samples", op="fork", code="e4m3", share=True, n=8, times=7, layers=2, Hkv=8, d=128, page=64,
             lo=1000, hi=32767),
        # whole copies of four sequences (sessions that will be evicted apart)
        dict(name="copy_sessions", op="fork", code="int8", share=False, n=4, times=1, layers=2, Hkv=8, d=128, page=64,
             lo=5001, hi=20000),
        # a forked branch of four long sequences evicted to a tenth, four layers
        dict(name="compact_branch_e4m3", op="compact", code="e4m3", n=4, layers=4, Hkv=4, d=128, page=64, lo=32768,
             hi=65535, kept_pct=10),
        # a small branch, half of it kept
        dict(name="compact_small_int8", op="compact", code="int8", n=2, layers=1, Hkv=8, d=96, page=32, lo=77, hi=1500,
             kept_pct=50),
    ]


def _log(rng, lo, hi):
    """An integer spread evenly over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """One more case: the same operators, sizes spread over their ranges, each
    within the largest listed case's work."""
    op = rng.choice(["attention", "attention", "store", "window", "fork", "compact"])
    code = rng.choice(["e4m3", "int8"])
    Hkv, g = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([1, 2, 3, 4, 6, 7, 8])
    d, page = rng.choice([16, 40, 64, 72, 80, 96, 112, 128]), rng.choice([32, 64, 128])
    if op == "attention":
        n = _log(rng, 1, 96)
        hi = _log(rng, 1, max(16, min(131072, 134217728 // (n * Hkv * d))))
        windowed = rng.random() < 0.4
        return dict(op=op, code=code, n=n, Hq=Hkv * g, Hkv=Hkv, d=d, page=page, T=rng.choice([1, 1, 1, 2, 3, 5, 8]),
                    lo=rng.randint(0, hi), hi=hi, window=_log(rng, 1, 8192) if windowed else 0,
                    sinks=rng.choice([0, 1, 4, 33, 130]) if windowed else 0)
    if op == "store":
        n = _log(rng, 1, 96)
        rows = _log(rng, 1, max(1, min(20000, 50000000 // (n * Hkv * d))))
        return dict(op=op, code=code, n=n, Hkv=Hkv, d=d, page=page, lo=rng.randint(1, rows), hi=rows,
                    old=rng.choice([0, 1]), rows=rows)
    if op == "window":
        Hq, B = Hkv * g, rng.choice([1, 1, 2, 3, 5])
        n = _log(rng, 1, max(64, min(20000, int(math.sqrt(1.5e9 / (B * Hq))))))
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, d=d, n=n, lo=rng.randint(0, n), window=_log(rng, 1, n + 5),
                    sinks=rng.choice([0, 1, 4, 64, 130]))
    layers = rng.choice([1, 2, 3])
    n = _log(rng, 1, 12)
    hi = _log(rng, 1, max(16, min(60000, 100000000 // (n * layers * Hkv * d))))
    lo = rng.randint(1, hi)
    if op == "fork":
        share = rng.random() < 0.5
        return dict(op=op, code=code, share=share, n=n, times=rng.randint(1, 5) if share else 1, layers=layers, Hkv=Hkv,
                    d=d, page=page, lo=lo, hi=hi)
    return dict(op=op, code=code, n=n, layers=layers, Hkv=Hkv, d=d, page=page, lo=lo, hi=hi,
                kept_pct=rng.randint(1, 100))


def _spread(lo, hi, n):
    """n lengths from lo to hi, the longest first."""
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _store_lengths(case):
    """(tokens already held, tokens to store) per sequence."""
    new = _spread(min(case["lo"], case["rows"]), min(case["hi"], case["rows"]), case["n"])
    if not case["old"]:
        return [0] * case["n"], new
    old = _spread(case["lo"], case["hi"], case["n"])
    return old, new


def _kept(case):
    return [max(0, length * case["kept_pct"] // 100) for length in _spread(case["lo"], case["hi"], case["n"])]


def _visible(length, T, window, sinks):
    """Tokens of a sequence that at least one of its last T rows sees, and the
    (row, token) pairs."""
    pairs, first = 0, 0
    for t in range(T):
        i = length - T + t
        if i < 0:
            continue
        full = i + 1
        pairs += full if not window else min(full, window + min(sinks, max(0, full - window)))
    top = max(0, length - T)
    if length <= 0:
        return 0, 0
    first = max(0, top - window + 1) if window else 0
    return length - first + min(sinks if window else 0, first), pairs


def work(case):
    op = case["op"]
    if op == "attention":
        H, Hq, d, T, n = case["Hkv"], case["Hq"], case["d"], case["T"], case["n"]
        b, f = 4.0 * n * Hq * T * d, 0.0
        for length in _spread(case["lo"], case["hi"], n):
            tokens, pairs = _visible(length, T, case["window"], case["sinks"])
            pages = -(-tokens // case["page"])
            b += tokens * H * d * 2 + pages * (8 * H + 4)
            f += 4.0 * pairs * Hq * d
        return dict(bytes=b, flops=f)
    if op == "store":
        H, d, page = case["Hkv"], case["d"], case["page"]
        old, new = _store_lengths(case)
        tokens = sum(new)
        pages = sum((o + c - 1) // page - o // page + 1 for o, c in zip(old, new) if c)
        return dict(bytes=tokens * H * d * 6.0 + pages * (8 * H + 4), flops=4.0 * tokens * H * d)
    if op == "window":
        H, Hq, d, W = case["Hkv"], case["Hq"], case["d"], case["window"]
        b = f = 0.0
        for length in _spread(case["lo"], case["n"], case["B"]):
            b += length * d * 2.0 * (2 * Hq + 2 * H)
            inside = min(W, length)
            pairs = inside * (inside + 1) / 2 + (length - inside) * inside
            more = max(0, length - W)       # row W + r sees min(r + 1, sinks) first tokens besides its window
            s = min(case["sinks"], more)
            pairs += s * (s + 1) / 2 + (more - s) * s
            f += 4.0 * pairs * Hq * d
        return dict(bytes=b, flops=f)
    H, d, page, layers = case["Hkv"], case["d"], case["page"], case["layers"]
    lengths = _spread(case["lo"], case["hi"], case["n"])
    if op == "fork":
        if case["share"]:
            moved = sum(1 for x in lengths if x % page) * case["times"]
        else:
            moved = sum(-(-x // page) for x in lengths)
        entries = sum(-(-x // page) for x in lengths) * case["times"]
        return dict(bytes=moved * layers * H * (page * d * 2 + 8) * 2.0 + entries * 16.0, flops=0.0)
    kept = sum(_kept(case))
    return dict(bytes=kept * layers * H * (4.0 * d + 4) + sum(lengths) / page * 16.0, flops=2.0 * kept * layers * H * d)


# ------------------------------------------------------------------ inputs
class State:
    """What a program has in hand before the call."""

    def __init__(self, **kw):
        self.__dict__.update(kw)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _page_scale(amax, code):
    """The scale of a page of largest magnitude `amax` (float32)."""
    if code == "int8":
        return (amax / QMAX_INT8).clamp_min(SCALE_MIN)
    m, e = torch.frexp(amax)                        # amax = m 2^e, 1/2 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.zeros_like(amax)).clamp_min(SCALE_MIN)


def _encode(x, code):
    """Codes of values already divided by their scale."""
    return x.round().clamp(-127, 127).to(torch.int8) if code == "int8" else x.to(torch.float8_e4m3fn)


def _cache(case, seed, lengths, seqs, spare, layers=1):
    """A pool as it is after some serving: pages in random order, keys with a
    few large channels, scales that differ from page to page.  `spare` pages
    stay free; sequences past len(lengths) are empty."""
    g, code = _gen(seed), case["code"]
    H, d, page = case["Hkv"], case["d"], case["page"]
    counts = [-(-x // page) for x in lengths]
    used, P = sum(counts), sum(counts) + spare
    M = max(1, max(counts))
    order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    table = torch.full((seqs, M), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(P, dtype=torch.int32, device="cuda")
    refs[order[:used].long()] = 1
    at = 0
    for i, c in enumerate(counts):
        table[i, :c] = order[at:at + c]
        at += c
    kv = []
    for which in range(2):
        codes = torch.empty(layers, P, H, page, d, dtype=torch.int8 if code == "int8" else torch.float8_e4m3fn,
                            device="cuda")
        scales = torch.empty(layers, P, H, dtype=torch.float32, device="cuda")
        for layer in range(layers):
            x = torch.randn(P, H, page, d, generator=g, device="cuda")
            if which == 0:
                x[..., :2] *= 3.0
            x *= torch.exp(0.5 * torch.randn(P, H, 1, 1, generator=g, device="cuda"))
            scales[layer] = _page_scale(x.abs().amax((2, 3)), code)
            codes[layer] = _encode(x / scales[layer][:, :, None, None], code)
        kv += [codes, scales]
    count = _ints(counts + [0] * (seqs - len(counts)))
    length = _ints(list(lengths) + [0] * (seqs - len(lengths)))
    s = State(case=case, code=code, layers=layers, P=P, M=M, k=kv[0], k_scale=kv[1], v=kv[2], v_scale=kv[3], refs=refs,
              table=table, count=count, length=length)
    return s


def _handle(s, seqs, Hq, T):
    """The package's cache holding the same contents."""
    from kv_cache_eviction_dropkv_gb300 import PagedCache

    c = s.case
    cache = PagedCache(seqs=seqs, Hkv=c["Hkv"], d=c["d"], pages=s.P, page=c["page"], max_pages=s.M, layers=s.layers,
                       code=s.code, Hq=Hq, T=T, device="cuda")
    for name in ("k", "v", "k_scale", "v_scale", "refs", "table", "count", "length"):
        getattr(cache, name).copy_(getattr(s, name))
        setattr(s, name, getattr(cache, name))
    s.cache = cache


def _spoil_tail(s):
    """Slots behind each sequence's last token hold whatever was there: not-a-number codes in e4m3."""
    if s.code != "e4m3":
        return
    page = s.case["page"]
    seq = (s.count > 0).nonzero()[:, 0]
    last = s.count[seq].long() - 1
    pg = s.table[seq, last].long()
    behind = last[:, None] * page + torch.arange(page, device="cuda") >= s.length[seq][:, None]
    for pool in (s.k, s.v):
        raw = pool.view(torch.uint8)
        rows = raw[0, pg]                                                     # [n][H][page][d]
        raw[0, pg] = torch.where(behind[:, None, :, None], torch.full_like(rows, 0x7F), rows)


def prepare(case, seed):
    op = case["op"]
    if op == "window":
        g = _gen(seed)
        B, Hq, H, d, n = case["B"], case["Hq"], case["Hkv"], case["d"], case["n"]
        q = torch.randn(B, Hq, n, d, generator=g, device="cuda").bfloat16()
        k = torch.randn(B, H, n, d, generator=g, device="cuda").bfloat16()
        v = torch.randn(B, H, n, d, generator=g, device="cuda").bfloat16()
        lengths = _ints(_spread(case["lo"], n, B))
        behind = (torch.arange(n, device="cuda") >= lengths[:, None])[:, None, :, None]
        k.masked_fill_(behind, float("nan"))
        v.masked_fill_(behind, float("nan"))
        s = State(case=case, q=q, k=k, v=v, lengths=lengths, out=torch.zeros_like(q))
        if own:
            from kv_cache_eviction_dropkv_gb300 import DropKV

            s.op = DropKV(B, Hq, H, d, n, 1, out_rows=1, device="cuda")
        return s
    if op == "attention":
        lengths = _spread(case["lo"], case["hi"], case["n"])
        s = _cache(case, seed, lengths, case["n"], 3)
        _spoil_tail(s)
        s.q = torch.randn(case["n"], case["Hq"], case["T"], case["d"], generator=_gen(seed + 1), device="cuda").bfloat16()
        s.out = torch.zeros_like(s.q)
        if own:
            _handle(s, case["n"], case["Hq"], case["T"])
        return s
    if op == "store":
        old, new = _store_lengths(case)
        s = _cache(case, seed, [a + b for a, b in zip(old, new)], case["n"], 3)
        g = _gen(seed + 1)
        shape = (case["n"], case["Hkv"], case["rows"], case["d"])
        s.src_k = (2.0 * torch.randn(shape, generator=g, device="cuda")).bfloat16()
        s.src_v = torch.randn(shape, generator=g, device="cuda").bfloat16()
        s.new = _ints(new)
        if own:
            _handle(s, case["n"], case["Hkv"], 1)
        return s
    lengths = _spread(case["lo"], case["hi"], case["n"])
    counts = [-(-x // case["page"]) for x in lengths]
    n = case["n"]
    if op == "fork":
        spare = (n * case["times"] if case["share"] else sum(counts)) + 5
        s = _cache(case, seed, lengths, n * (1 + case["times"]), spare, case["layers"])
        s.src = _ints([i for i in range(n) for _ in range(case["times"])])
        s.dst = _ints([n + i for i in range(n * case["times"])])
        if own:
            _handle(s, n * (1 + case["times"]), case["Hkv"], 1)
        return s
    kept = _kept(case)
    s = _cache(case, seed, lengths, 2 * n, n + sum(-(-x // case["page"]) for x in kept) + 5, case["layers"])
    s.src, s.dst = _ints(list(range(n))), _ints(list(range(n, 2 * n)))
    s.kept_len = _ints(kept)
    g = _gen(seed + 1)
    s.kept_idx = torch.zeros(case["layers"], n, case["Hkv"], max(1, max(kept)), dtype=torch.int32, device="cuda")
    for i, (length, m) in enumerate(zip(lengths, kept)):
        lot = torch.rand(case["layers"], case["Hkv"], length, generator=g, device="cuda").argsort(-1)[..., :m]
        s.kept_idx[:, i, :, :m] = lot.sort(-1).values.to(torch.int32)
    if own:
        _handle(s, 2 * n, case["Hkv"], 1)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return {"attention": _attention, "store": _store, "window": _window, "fork": _fork, "compact": _compact}[
        s.case["op"]](s)


def _buffers(s):
    return dict(k=s.k, v=s.v, k_scale=s.k_scale, v_scale=s.v_scale, refs=s.refs, table=s.table, count=s.count,
                length=s.length)


def _values(s, layer, pages):
    """K and V values of table entries `pages` [n][M]: [n][Hkv][M * page][d] float32."""
    got = []
    for codes, scale in ((s.k, s.k_scale), (s.v, s.v_scale)):
        raw = codes[layer].view(torch.uint8)[pages].view(codes.dtype)
        x = raw.to(torch.float32) * scale[layer][pages][..., None, None]
        n, M, H, page, d = x.shape
        got.append(x.permute(0, 2, 1, 3, 4).reshape(n, H, M * page, d))
    return got


def _softmax_rows(x, v):
    """softmax(x) v over the last axis of x, 0 for rows without a finite logit."""
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    return torch.where(total > 0, p @ v / total, torch.zeros((), device=x.device, dtype=x.dtype))


def _attention(s):
    c = s.case
    if own:
        s.cache.attention(0, s.q, s.out, window=c["window"], sinks=c["sinks"])
        return s.out
    n, Hq, H, T, d = c["n"], c["Hq"], c["Hkv"], c["T"], c["d"]
    k, v = _values(s, 0, s.table.clamp_min(0).long())
    j = torch.arange(k.shape[2], device="cuda")
    i = s.length[:, None].long() - T + torch.arange(T, device="cuda")                     # [n][T]
    seen = j <= i[..., None]
    if c["window"]:
        seen &= (j < c["sinks"]) | (j > i[..., None] - c["window"])
    v = torch.where((j < s.length[:, None])[:, None, :, None], v, torch.zeros((), device="cuda"))
    q = s.q.float().reshape(n, H, Hq // H * T, d)
    x = q @ k.transpose(-1, -2) / math.sqrt(d)
    x = x.reshape(n, H, Hq // H, T, -1).masked_fill(~seen[:, None, None], -math.inf)
    o = _softmax_rows(x.reshape(n, H, Hq // H * T, -1), v)
    s.out.copy_(o.reshape(n, Hq, T, d))
    return s.out


def _store(s):
    c = s.case
    if own:
        s.cache.store(0, s.src_k, s.src_v, s.new)
        return dict(k=s.k, v=s.v, k_scale=s.k_scale, v_scale=s.v_scale)
    page, code = c["page"], s.code
    start = (s.length - s.new).long()
    cols = (start // page)[:, None] + torch.arange((c["rows"] + page - 2) // page + 1, device="cuda")  # touched pages
    live = (cols < s.count[:, None]) & (s.new > 0)[:, None]
    seq, col = live.nonzero(as_tuple=True)
    pg = s.table[seq, cols[seq, col]].long()
    pos = cols[seq, col][:, None] * page + torch.arange(page, device="cuda")
    row = pos - start[seq][:, None]
    new = (row >= 0) & (row < s.new[seq][:, None])
    old = row < 0
    for src, codes, scales in ((s.src_k, s.k, s.k_scale), (s.src_v, s.v, s.v_scale)):
        x = src.transpose(1, 2)[seq[:, None], row.clamp(0, c["rows"] - 1)].float().transpose(1, 2)   # [pages][H][page][d]
        fresh = _page_scale(torch.where(new[:, None, :, None], x.abs(), torch.zeros((), device="cuda")).amax((2, 3)), code)
        held = scales[0][pg]
        scale = torch.where(old.any(-1)[:, None], torch.maximum(held, fresh), fresh)
        was = codes[0].view(torch.uint8)[pg].view(codes.dtype)
        again = _encode(was.float() * held[..., None, None] / scale[..., None, None], code)
        put = _encode(x / scale[..., None, None], code)
        keep = torch.where(old[:, None, :, None], again.view(torch.uint8), was.view(torch.uint8))
        codes[0].view(torch.uint8)[pg] = torch.where(new[:, None, :, None], put.view(torch.uint8), keep)
        scales[0][pg] = scale
    return dict(k=s.k, v=s.v, k_scale=s.k_scale, v_scale=s.v_scale)


def _window(s):
    c = s.case
    if own:
        s.op.window_attention(s.q, s.k, s.v, s.lengths, s.out, c["window"], c["sinks"])
        return s.out
    B, Hq, H, d, n, S = c["B"], c["Hq"], c["Hkv"], c["d"], c["n"], min(c["sinks"], c["n"])
    W = min(c["window"], n)
    blocks = -(-n // W)                                    # blocks of W rows, each against its own and the block before
    inside = (torch.arange(n, device="cuda") < s.lengths[:, None])[:, None, :, None]
    k, v = (torch.where(inside, x.float(), torch.zeros((), device="cuda")) for x in (s.k, s.v))
    pad = blocks * W - n
    more = W if blocks > 1 else 0

    def spans(x):
        x = torch.nn.functional.pad(x, (0, 0, more, pad)).reshape(B, H, -1, W, d)
        return torch.cat((x[:, :, :-1], x[:, :, 1:]), 3) if more else x

    q = torch.nn.functional.pad(s.q.float(), (0, 0, 0, pad)).reshape(B, H, Hq // H, blocks, W, d)
    q = q.transpose(2, 3).reshape(B, H, blocks, Hq // H * W, d)
    i = torch.arange(W, device="cuda")[:, None]
    j = torch.arange(W + more, device="cuda") - more       # key minus the block's first row
    near = (j <= i) & (j > i - W)
    first = torch.arange(blocks, device="cuda")[:, None, None] * W
    near = near & (j + first >= 0)                         # [blocks][W][span]
    far = (torch.arange(S, device="cuda") <= i + first - W)   # first tokens outside the window
    x = torch.cat((q @ spans(k).transpose(-1, -2), q @ k[:, :, None, :S].transpose(-1, -2)), -1).div_(math.sqrt(d))
    seen = torch.cat((near, far), -1)
    x = x.reshape(B, H, blocks, Hq // H, W, -1).masked_fill_(~seen[:, None], -math.inf)
    x = x.reshape(B, H, blocks, Hq // H * W, -1)
    x.sub_(x.amax(-1, keepdim=True)).exp_()                # a row sees itself at least
    total = x.sum(-1, keepdim=True)
    o = x[..., :W + more] @ spans(v) + x[..., W + more:] @ v[:, :, None, :S]
    o = (o / total).reshape(B, H, blocks, Hq // H, W, d).transpose(2, 3).reshape(B, Hq, blocks * W, d)[:, :, :n]
    s.out.copy_(torch.where(inside, o.to(torch.bfloat16), s.out))
    return s.out


def _plain_free(s, seqs):
    held = s.table[seqs]
    live = torch.arange(s.M, device="cuda") < s.count[seqs][:, None]
    s.refs.index_add_(0, held.clamp_min(0).flatten().long(), -live.flatten().to(torch.int32))
    s.table[seqs] = -1
    s.count[seqs] = 0
    s.length[seqs] = 0


def _plain_take(s, wanted):
    """The lowest free pages for the true entries of `wanted` [n][M], in order; -1 elsewhere."""
    free_first = torch.argsort((s.refs != 0).to(torch.int32), stable=True).to(torch.int32)
    rank = wanted.flatten().cumsum(0) - 1
    taken = free_first[rank.clamp_min(0)].reshape(wanted.shape)
    s.refs.index_add_(0, taken.flatten().long(), wanted.flatten().to(torch.int32))
    return torch.where(wanted, taken, torch.full_like(taken, -1))


def _plain_fork(s, src, dst, share):
    col = torch.arange(s.M, device="cuda")
    held, count = s.table[src], s.count[src][:, None]
    whole = (s.length[src] // s.case["page"])[:, None] if share else torch.zeros_like(count)
    shared, fresh = col < whole, (col >= whole) & (col < count)
    s.refs.index_add_(0, held.clamp_min(0).flatten().long(), shared.flatten().to(torch.int32))
    taken = _plain_take(s, fresh)
    a, b = held[fresh].long(), taken[fresh].long()
    for codes, scales in ((s.k, s.k_scale), (s.v, s.v_scale)):
        codes.view(torch.uint8)[:, b] = codes.view(torch.uint8)[:, a]
        scales[:, b] = scales[:, a]
    s.table[dst] = torch.where(shared, held, taken)
    s.count[dst] = s.count[src]
    s.length[dst] = s.length[src]


def _fork(s):
    """The forks of the pass before end, and new ones are made."""
    share = s.case["share"]
    if own:
        s.cache.free(s.dst)
        (s.cache.fork if share else s.cache.copy)(s.src, s.dst)
    else:
        _plain_free(s, s.dst.long())
        _plain_fork(s, s.src.long(), s.dst.long(), share)
    return _buffers(s)


def _compact(s):
    """The branch of the pass before ends; a new one is forked and evicted."""
    if own:
        s.cache.free(s.dst)
        s.cache.fork(s.src, s.dst)
        s.cache.compact(s.kept_idx, s.kept_len, s.dst)
        return _buffers(s)
    page = s.case["page"]
    src, dst = s.src.long(), s.dst.long()
    _plain_free(s, dst)
    _plain_fork(s, src, dst, True)
    held = s.table[dst].long()                                                 # [n][M]
    pages = (s.kept_len + page - 1) // page
    wanted = torch.arange(s.M, device="cuda") < pages[:, None]
    taken = _plain_take(s, wanted)
    seq, col = wanted.nonzero(as_tuple=True)
    pg = taken[seq, col].long()
    slot = col[:, None] * page + torch.arange(page, device="cuda")             # [new pages][page]
    live = slot < s.kept_len[seq][:, None]
    idx = s.kept_idx[:, seq].long()                                            # [layers][new pages][H][kept]
    idx = idx.gather(-1, slot.clamp_max(idx.shape[-1] - 1)[None, :, None].expand(idx.shape[0], -1, idx.shape[2], -1))
    idx = torch.where(live[:, None], idx, torch.zeros_like(idx))
    old = held[seq[:, None, None], idx // page]                                # [layers][new pages][H][page]
    layer = torch.arange(s.layers, device="cuda")[:, None, None, None]
    head = torch.arange(s.case["Hkv"], device="cuda")[:, None]
    for codes, scales in ((s.k, s.k_scale), (s.v, s.v_scale)):
        was = scales[layer, old, head]
        scale = torch.where(live[:, None], was, torch.zeros_like(was)).amax(-1)
        raw = codes.view(torch.uint8)
        x = raw[layer, old, head, idx % page].view(codes.dtype).float() * was[..., None] / scale[..., None, None]
        put = torch.where(live[:, None, :, None], _encode(x, s.code).view(torch.uint8), raw[:, pg])
        raw[:, pg] = put
        scales[:, pg] = scale
    there = torch.arange(s.M, device="cuda") < s.count[dst][:, None]
    s.refs.index_add_(0, held.clamp_min(0).flatten(), -there.flatten().to(torch.int32))
    s.table[dst] = taken
    s.count[dst] = pages
    s.length[dst] = s.kept_len
    return _buffers(s)


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_scale(amax, code):
    """The page scale from the largest magnitude, a Python float (0: an empty page)."""
    if code == "int8":
        # the scale is a 32-bit number by definition
        return max(float(torch.tensor(amax, dtype=torch.float32) / 127), 2.0 ** -120)
    return max(2.0 ** math.ceil(math.log2(amax / 448.0)), 2.0 ** -120) if amax > 0 else 2.0 ** -120


def _exact_e4m3(x):
    """The nearest e4m3 value (ties to even), |x| <= 448, in float64."""
    e = torch.floor(torch.log2(x.abs().clamp_min(1e-300))).clamp_min(-6.0)
    step = torch.exp2(e - 3.0)
    return torch.round(x / step) * step


def exact(case, seed):
    op = case["op"]
    global own
    mine, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = mine
    if op == "attention":
        n, Hq, H, T, d, page = case["n"], case["Hq"], case["Hkv"], case["T"], case["d"], case["page"]
        out = torch.zeros(n, Hq, T, d, dtype=torch.float64, device="cuda")
        for b, L in enumerate(s.length.tolist()):
            pages = s.table[b, :-(-L // page)].long()
            kk, vv = (c[0].view(torch.uint8)[pages].view(c.dtype).double() * sc[0][pages].double()[..., None, None]
                      for c, sc in ((s.k, s.k_scale), (s.v, s.v_scale)))
            for h in range(H):
                k, v = kk[:, h].reshape(-1, d)[:L], vv[:, h].reshape(-1, d)[:L]
                for t in range(T):
                    i = L - T + t
                    if i < 0:
                        continue
                    lo = max(0, i - case["window"] + 1) if case["window"] else 0
                    head = min(case["sinks"], lo) if case["window"] else 0
                    ks, vs = (torch.cat((a[:head], a[lo:i + 1])) for a in (k, v))
                    q = s.q[b, h * (Hq // H):(h + 1) * (Hq // H), t].double()
                    out[b, h * (Hq // H):(h + 1) * (Hq // H), t] = torch.softmax(q @ ks.T / math.sqrt(d), -1) @ vs
        return out
    if op == "window":
        B, Hq, H, d, W, S = case["B"], case["Hq"], case["Hkv"], case["d"], case["window"], case["sinks"]
        if case["Hq"] * case["n"] * min(case["n"], W + 1024) * B * d > 2e12:
            return None
        out = torch.zeros(B, Hq, case["n"], d, dtype=torch.float64, device="cuda")
        for b, L in enumerate(s.lengths.tolist()):
            for h in range(H):
                for i0 in range(0, L, 1024):
                    i1 = min(L, i0 + 1024)
                    lo = max(0, i0 - W + 1)
                    j = torch.cat((torch.arange(min(S, lo)), torch.arange(lo, i1))).cuda()
                    i = torch.arange(i0, i1, device="cuda")[:, None]
                    hide = (j > i) | ((j <= i - W) & (j >= S))
                    k, v = s.k[b, h][j].double(), s.v[b, h][j].double()
                    for hq in range(h * Hq // H, (h + 1) * Hq // H):
                        x = s.q[b, hq, i0:i1].double() @ k.T / math.sqrt(d)
                        out[b, hq, i0:i1] = torch.softmax(x.masked_fill_(hide, -math.inf), -1) @ v
        return out
    if op == "store":
        old, new = _store_lengths(case)
        page, res = case["page"], {}
        if sum(new) * case["Hkv"] > 2000000:
            return None
        for name, src, codes, scales in (("k", s.src_k, s.k, s.k_scale), ("v", s.src_v, s.v, s.v_scale)):
            codes, scales = codes.double(), scales.double()
            for b, (o, c) in enumerate(zip(old, new)):
                for col in range(o // page, -(-(o + c) // page) if c else 0):
                    pg = int(s.table[b, col])
                    a, z = max(o, col * page), min(o + c, (col + 1) * page)        # new positions of this page
                    x = src[b, :, a - o:z - o].double()
                    top = x.abs().amax((1, 2)).tolist()
                    for h, t in enumerate(top):
                        was = float(scales[0, pg, h])
                        sc = max(_exact_scale(t, case["code"]), was if a > col * page else 0.0)
                        if case["code"] == "e4m3":
                            codes[0, pg, h, :a - col * page] = _exact_e4m3(codes[0, pg, h, :a - col * page] * was / sc)
                            codes[0, pg, h, a - col * page:z - col * page] = _exact_e4m3(x[h] / sc)
                        scales[0, pg, h] = sc
            res[name] = codes if case["code"] == "e4m3" else None
            res[name + "_scale"] = scales
        return res
    # pages: which page numbers are taken follows from the counts; the contents are those of the sequences
    page, n = case["page"], case["n"]
    free = [p for p, r in enumerate(s.refs.tolist()) if r == 0]
    table, lengths = s.table.tolist(), s.length.tolist()
    res = dict(k=s.k.double(), v=s.v.double(), k_scale=s.k_scale.double(), v_scale=s.v_scale.double())
    branch = {}
    at = 0
    for src, dst in zip(s.src.tolist(), s.dst.tolist()):
        L = lengths[src]
        pages = table[src][:-(-L // page)]
        first = L // page if op == "compact" or case["share"] else 0
        branch[dst] = list(pages)
        for col in range(first, len(pages)):
            to = free[at]
            at += 1
            for x in res.values():
                x[:, to] = x[:, pages[col]]
            branch[dst][col] = to
    if op == "compact":
        for b, (dst, m) in enumerate(zip(s.dst.tolist(), s.kept_len.tolist())):
            for col in range(-(-m // page)):
                to = free[at]
                at += 1
                idx = s.kept_idx[:, b, :, col * page:min(m, (col + 1) * page)].long()      # [layers][H][tokens]
                frm = torch.tensor(branch[dst], device="cuda")[idx // page]
                la = torch.arange(idx.shape[0], device="cuda")[:, None, None]
                hd = torch.arange(idx.shape[1], device="cuda")[:, None]
                for name in ("k", "v"):
                    was = res[name + "_scale"][la, frm, hd]
                    top = was.amax(-1)
                    x = res[name][la, frm, hd, idx % page] * (was / top[..., None])[..., None]
                    res[name][:, to, :, :idx.shape[2]] = _exact_e4m3(x) if case["code"] == "e4m3" else x
                    res[name + "_scale"][:, to] = top
    if case["code"] == "int8":
        res["k"] = res["v"] = None
    res.update(refs=None, table=None, count=None, length=None)
    return res
