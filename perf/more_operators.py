"""Workloads of what surrounds the paged 8-bit cache in a serving step.

Each case is one call a program makes next to `perf/operators.py`'s: queries
and keys get their per-head norm and their positions (a prompt's, or a decode
step's with the keys and values stored in the same call), a sequence's codes
are read back as bf16 rows for another scoring, and forked sequences attend
over the pages they share once for all.  `own` selects the package's kernels;
otherwise the same pass is computed in its plain form, elementary torch
operations in 32 bits rounded once at the end.  `exact` computes the outputs
from the definitions in 64 bits.

Rotation: pair i of the first `dims` channels of a head (channels i and i +
dims / 2, or 2 i and 2 i + 1) turns by position * freq_i; freq_i =
base^(-2 i / dims), changed by the scaling that a long context asks for.  The
norm before it is x / sqrt(mean(x^2) + eps) * weight over the head.  The cache
is that of `perf/operators.py`: codes [layers][pages][Hkv][page][d] in e4m3 or
int8, one scale per page and KV head, value = code * scale.
"""
import math

import torch

own = False

SCALE_MIN = 2.0 ** -120      # smallest scale of a page
EPS = 1e-6
SCALINGS = {
    "none": None,
    "linear": dict(kind="linear", factor=4.0),
    "ntk": dict(kind="ntk", factor=8.0),
    "yarn": dict(kind="yarn", factor=16.0, original=4096),
    "bands": dict(kind="bands", factor=8.0, original=8192),
}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step of 64 sequences deep in their contexts: one token's queries and keys, normed and turned; latency
        dict(name="rotate_step", op="rotate", B=64, Hq=32, Hkv=8, d=128, dims=128, layout="half", norm=True,
             scaling="bands", base=500000.0, n=1, lo=1, first=131072, packed=True),
        # a 32K prompt out of its packed projection into the layout that attention and scoring read
        dict(name="rotate_prompt_32k", op="rotate", B=1, Hq=32, Hkv=8, d=128, dims=128, layout="half", norm=True,
             scaling="none", base=1000000.0, n=32768, lo=32768, first=0, packed=True),
        # a padded batch of MHA prompts with d = 96, half of each head turned, pairs side by side, a stretched context
        dict(name="rotate_batch_partial", op="rotate", B=4, Hq=32, Hkv=32, d=96, dims=48, layout="interleaved",
             norm=False, scaling="yarn", base=10000.0, n=2051, lo=700, first=60000, packed=False),
        # one decode step of 64 sequences straight into the cache
        dict(name="store_rotated_step", op="store", n=64, Hq=32, Hkv=8, d=128, page=64, dims=128, layout="half",
             norm=True, scaling="none", base=1000000.0, lo=1, hi=4095, rows=1, old=1, packed=True),
        # chunks of four prompts behind what their sequences hold
        dict(name="store_rotated_chunk", op="store", n=4, Hq=32, Hkv=8, d=128, page=64, dims=64, layout="half",
             norm=True, scaling="linear", base=10000.0, lo=1000, hi=8192, rows=8192, old=1, packed=True),
        # a sequence of the headline length read back, to be scored again
        dict(name="read_rescore_128k", op="read", code="e4m3", n=1, Hkv=8, d=128, page=64, lo=131072, hi=131072,
             tail=131072),
        # the newest 500 tokens of a ragged batch, int8 codes, d = 96
        dict(name="read_newest_int8", op="read", code="int8", n=24, Hkv=4, d=96, page=128, lo=300, hi=9000, tail=500),
        # eight samples of one short prompt, a few tokens in; latency
        dict(name="shared_samples_first", op="shared", code="e4m3", groups=1, mlo=8, mhi=8, Hq=32, Hkv=8, d=128, page=64,
             T=1, plo=1000, phi=1000, lo=1, hi=64),
        # 64 conversations behind one long system prompt
        dict(name="shared_system_prompt", op="shared", code="e4m3", groups=1, mlo=64, mhi=64, Hq=32, Hkv=8, d=128,
             page=64, T=1, plo=32768, phi=32768, lo=1, hi=2000),
        # eight prompts of the 28/4-head layer sampled 1 to 12 times each, int8 codes
        dict(name="shared_groups_int8", op="shared", code="int8", groups=8, mlo=1, mhi=12, Hq=28, Hkv=4, d=128, page=128,
             T=1, plo=1000, phi=30000, lo=1, hi=1000),
        # two MHA prompts with d = 96, twelve samples each, four drafted tokens a step
        dict(name="shared_draft_mha", op="shared", code="e4m3", groups=2, mlo=12, mhi=12, Hq=32, Hkv=32, d=96, page=32,
             T=4, plo=2000, phi=6001, lo=5, hi=500),
        # sixteen questions about one document of the headline length
        dict(name="shared_document_128k", op="shared", code="e4m3", groups=1, mlo=16, mhi=16, Hq=32, Hkv=8, d=128,
             page=64, T=1, plo=131072, phi=131072, lo=10, hi=300),
    ]


def _log(rng, lo, hi):
    """An integer spread evenly over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """One more case: the same operators, sizes spread over their ranges, each
    within the largest listed case's work."""
    op = rng.choice(["rotate", "store", "read", "shared", "shared"])
    Hkv, g = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([1, 2, 3, 4, 6, 7, 8])
    d, page = rng.choice([16, 40, 64, 72, 80, 96, 112, 128]), rng.choice([32, 64, 128])
    turned = dict(dims=rng.choice([x for x in (8, 16, 24, 32, 40, 64, 96, 128) if x < d] + [d] * 3),
                  layout=rng.choice(["half", "interleaved"]), norm=rng.random() < 0.5,
                  scaling=rng.choice(sorted(SCALINGS)), base=rng.choice([10000.0, 500000.0, 1000000.0]))
    if op == "rotate":
        B = _log(rng, 1, 96)
        n = _log(rng, 1, max(1, min(32768, 150000000 // (B * (g + 1) * Hkv * d))))
        return dict(op=op, B=B, Hq=Hkv * g, Hkv=Hkv, d=d, **turned, n=n, lo=rng.randint(0, n),
                    first=rng.choice([0, 17, 131072, 1000000]), packed=rng.random() < 0.6)
    if op == "store":
        n = _log(rng, 1, 96)
        rows = _log(rng, 1, max(1, min(16384, 60000000 // (n * (g + 2) * Hkv * d))))
        return dict(op=op, n=n, Hq=Hkv * g, Hkv=Hkv, d=d, page=page, **turned, lo=rng.randint(1, rows), hi=rows,
                    rows=rows, old=rng.choice([0, 1]), packed=rng.random() < 0.6)
    code = rng.choice(["e4m3", "int8"])
    if op == "read":
        n = _log(rng, 1, 96)
        hi = _log(rng, 1, max(16, min(131072, 134217728 // (n * Hkv * d))))
        return dict(op=op, code=code, n=n, Hkv=Hkv, d=d, page=page, lo=rng.randint(0, hi), hi=hi,
                    tail=_log(rng, 1, hi))
    groups, T = _log(rng, 1, 12), rng.choice([1, 1, 1, 2, 3, 5])
    mhi = _log(rng, 1, max(1, 96 // groups))
    total = max(64, min(131072, 1000000000 // (groups * mhi * Hkv * d)))
    phi = _log(rng, 1, total)
    return dict(op=op, code=code, groups=groups, mlo=rng.randint(1, mhi), mhi=mhi, Hq=Hkv * g, Hkv=Hkv, d=d, page=page,
                T=T, plo=rng.randint(0, phi), phi=phi, lo=rng.randint(0, 40), hi=40 + _log(rng, 1, 1500))


def _spread(lo, hi, n):
    """n numbers from lo to hi, the largest first."""
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _stored(case):
    """(tokens already held, tokens to store) per sequence."""
    new = _spread(case["lo"] if case["lo"] < case["rows"] else case["rows"], min(case["hi"], case["rows"]), case["n"])
    return (_spread(case["lo"], case["hi"], case["n"]) if case["old"] else [0] * case["n"]), new


def _shared(case):
    """Per group: (tokens of the prefix, tokens of each member)."""
    sizes = _spread(case["mlo"], case["mhi"], case["groups"])
    return [(p, [p + x for x in _spread(case["lo"], case["hi"], m)])
            for p, m in zip(_spread(case["plo"], case["phi"], case["groups"]), sizes)]


def _newest(case):
    """(first token, tokens) that are read back of each sequence."""
    lengths = _spread(case["lo"], case["hi"], case["n"])
    return [max(0, x - case["tail"]) for x in lengths], [min(x, case["tail"]) for x in lengths]


def work(case):
    op, H, d = case["op"], case["Hkv"], case["d"]
    if op == "rotate":
        tokens = sum(_spread(case["lo"], case["n"], case["B"]))
        rows = tokens * (case["Hq"] + H)
        return dict(bytes=rows * d * 4.0, flops=rows * (3.0 * case["dims"] + (4.0 * d if case["norm"] else 0.0)))
    if op == "store":
        old, new = _stored(case)
        tokens, page = sum(new), case["page"]
        pages = sum((o + c - 1) // page - o // page + 1 for o, c in zip(old, new) if c)
        rows = tokens * (case["Hq"] + H)
        return dict(bytes=tokens * d * (6.0 * H + 4.0 * case["Hq"]) + pages * (8 * H + 4),
                    flops=rows * (3.0 * case["dims"] + (4.0 * d if case["norm"] else 0.0)) + 4.0 * tokens * H * d)
    if op == "read":
        tokens = sum(_newest(case)[1])
        return dict(bytes=tokens * H * d * 6.0 + tokens / case["page"] * (8 * H + 4), flops=2.0 * tokens * H * d)
    b = f = 0.0
    for prefix, lengths in _shared(case):
        whole = prefix // case["page"] * case["page"]
        tokens = whole + sum(x - whole for x in lengths)
        b += tokens * H * (2.0 * d + 8.0 / case["page"]) + 4.0 * len(lengths) * case["Hq"] * case["T"] * d
        f += sum(4.0 * max(0, x - t) * case["Hq"] * d for x in lengths for t in range(case["T"]))
    return dict(bytes=b, flops=f)


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
        return (amax / 127.0).clamp_min(SCALE_MIN)
    m, e = torch.frexp(amax)                        # amax = m 2^e, 1/2 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.zeros_like(amax)).clamp_min(SCALE_MIN)


def _encode(x, code):
    """Codes of values already divided by their scale."""
    return x.round().clamp(-127, 127).to(torch.int8) if code == "int8" else x.to(torch.float8_e4m3fn)


def _pool(case, seed, code, P, M, tables, lengths):
    """A pool as it is after some serving: keys with a few large channels,
    scales that differ from page to page, the given page tables."""
    g, H, d, page = _gen(seed), case["Hkv"], case["d"], case["page"]
    table = torch.full((len(tables), M), -1, dtype=torch.int32)
    refs = torch.zeros(P, dtype=torch.int32)
    for i, t in enumerate(tables):
        table[i, :len(t)] = t
        refs.index_add_(0, t.long(), torch.ones_like(t))
    kv = []
    for which in range(2):
        x = torch.randn(P, H, page, d, generator=g, device="cuda")
        if which == 0:
            x[..., :2] *= 3.0
        x *= torch.exp(0.5 * torch.randn(P, H, 1, 1, generator=g, device="cuda"))
        scale = _page_scale(x.abs().amax((2, 3)), code)
        kv += [_encode(x / scale[..., None, None], code)[None], scale[None]]
    return State(case=case, code=code, P=P, M=M, k=kv[0], k_scale=kv[1], v=kv[2], v_scale=kv[3], refs=refs.cuda(),
                 table=table.cuda(), count=_ints([len(t) for t in tables]), length=_ints(lengths))


def _apart(case, seed, code, lengths, spare):
    """Sequences that share no page, pages in random order."""
    counts = [-(-x // case["page"]) for x in lengths]
    g = torch.Generator()
    g.manual_seed(seed)
    order = torch.randperm(sum(counts) + spare, generator=g).to(torch.int32)
    tables, at = [], 0
    for c in counts:
        tables.append(order[at:at + c])
        at += c
    return _pool(case, seed, code, sum(counts) + spare, max(1, max(counts)), tables, lengths)


def _handle(s, Hq=None, T=1, groups=0):
    """The package's cache holding the same contents."""
    from kv_cache_eviction_dropkv_gb300 import PagedCache

    c = s.case
    cache = PagedCache(seqs=len(s.length), Hkv=c["Hkv"], d=c["d"], pages=s.P, page=c["page"], max_pages=s.M, layers=1,
                       code=s.code, Hq=Hq, T=T, groups=groups, device="cuda")
    for name in ("k", "v", "k_scale", "v_scale", "refs", "table", "count", "length"):
        getattr(cache, name).copy_(getattr(s, name))
        setattr(s, name, getattr(cache, name))
    s.cache = cache


def _spoil_tail(s):
    """Slots behind each sequence's last token hold whatever was there: not-a-number codes in e4m3."""
    if s.code != "e4m3":
        return
    page = s.case["page"]
    seq = (s.length % page > 0).nonzero()[:, 0]
    last = s.count[seq].long() - 1
    pg = s.table[seq, last].long()
    behind = last[:, None] * page + torch.arange(page, device="cuda") >= s.length[seq][:, None]
    for pool in (s.k, s.v):
        raw = pool.view(torch.uint8)
        rows = raw[0, pg]                                                     # [n][H][page][d]
        raw[0, pg] = torch.where(behind[:, None, :, None], torch.full_like(rows, 0x7F), rows)


def _weights(case, g):
    """Norm weights of queries and keys, or None."""
    if not case["norm"]:
        return None, None
    return tuple((1.0 + 0.3 * torch.randn(case["d"], generator=g, device="cuda")).bfloat16().float() for _ in range(2))


def _rotary(s):
    """The package's plan of the case's norm and rotation."""
    from kv_cache_eviction_dropkv_gb300 import Rotary

    c = s.case
    s.rotary = Rotary(c["d"], dims=c["dims"], base=c["base"], layout=c["layout"], scaling=SCALINGS[c["scaling"]],
                      q_norm=s.qw, k_norm=s.kw, eps=EPS, device="cuda")


def _projected(case, n, rows, g):
    """Queries, keys and values as a layer's projection leaves them: one row of
    (Hq + 2 Hkv) d numbers per token, or three tensors of the library's layout."""
    Hq, H, d = case["Hq"], case["Hkv"], case["d"]
    if case["packed"]:
        x = torch.randn(n, rows, Hq + 2 * H, d, generator=g, device="cuda").bfloat16()
        x[:, :, Hq:Hq + H, :2] *= 3.0
        return tuple(t.transpose(1, 2) for t in x.split((Hq, H, H), 2))
    q, k, v = (torch.randn(n, h, rows, d, generator=g, device="cuda").bfloat16() for h in (Hq, H, H))
    k[..., :2] *= 3.0
    return q, k, v


def prepare(case, seed):
    op = case["op"]
    if op == "rotate":
        g = _gen(seed)
        q, k, _ = _projected(case, case["B"], case["n"], g)
        qw, kw = _weights(case, g)
        first = torch.randint(case["first"] // 2, case["first"] + 1, (case["B"],), generator=g, device="cuda")
        s = State(case=case, q=q, k=k, qw=qw, kw=kw, positions=first.to(torch.int32),
                  lengths=_ints(_spread(case["lo"], case["n"], case["B"])),
                  q_out=torch.zeros(q.shape, dtype=q.dtype, device="cuda"),
                  k_out=torch.zeros(k.shape, dtype=k.dtype, device="cuda"))
        if own:
            _rotary(s)
        return s
    if op == "store":
        old, new = _stored(case)
        s = _apart(case, seed, "e4m3", [a + b for a, b in zip(old, new)], 3)
        g = _gen(seed + 1)
        s.q, s.src_k, s.src_v = _projected(case, case["n"], case["rows"], g)
        s.qw, s.kw = _weights(case, g)
        s.new, s.positions = _ints(new), _ints([3 * x for x in old])       # an evicted cache: positions run ahead of slots
        s.q_out = torch.zeros(s.q.shape, dtype=s.q.dtype, device="cuda")
        if own:
            _rotary(s)
            _handle(s, case["Hq"])
        return s
    if op == "read":
        s = _apart(case, seed, case["code"], _spread(case["lo"], case["hi"], case["n"]), 3)
        s.starts, s.counts = (_ints(x) for x in _newest(case))
        rows = max(1, int(s.counts.max()))
        s.k_out, s.v_out = (torch.zeros(case["n"], case["Hkv"], rows, case["d"], dtype=torch.bfloat16, device="cuda")
                            for _ in range(2))
        if own:
            _handle(s)
        return s
    parts, page = _shared(case), case["page"]
    lengths = [x for _, xs in parts for x in xs]
    P = sum(p // page + sum(-(-x // page) - p // page for x in xs) for p, xs in parts) + 3
    g = torch.Generator()
    g.manual_seed(seed)
    order, at, tables = torch.randperm(P, generator=g).to(torch.int32), 0, []
    for p, xs in parts:
        common = order[at:at + p // page]
        at += p // page
        for x in xs:
            more = -(-x // page) - p // page
            tables.append(torch.cat((common, order[at:at + more])))
            at += more
    s = _pool(case, seed, case["code"], P, max(1, max(len(t) for t in tables)), tables, lengths)
    _spoil_tail(s)
    starts = [0]
    for _, xs in parts:
        starts.append(starts[-1] + len(xs))
    s.groups = _ints(starts)
    s.q = torch.randn(len(lengths), case["Hq"], case["T"], case["d"], generator=_gen(seed + 1), device="cuda").bfloat16()
    s.out = torch.zeros_like(s.q)
    if own:
        _handle(s, case["Hq"], case["T"], case["groups"])
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return {"rotate": _rotate, "store": _store, "read": _read, "shared": _attention}[s.case["op"]](s)


def _frequencies(case):
    """Radians per position of each pair (float64), and the factor of the rotated channels."""
    dims, base, how = case["dims"], case["base"], SCALINGS[case["scaling"]]
    i = torch.arange(dims // 2, dtype=torch.float64, device="cuda")
    if how and how["kind"] == "ntk":
        base = base * how["factor"] ** (dims / max(1, dims - 2))
    freq = base ** (-2.0 * i / dims)
    if not how or how["kind"] == "ntk":
        return freq, 1.0
    if how["kind"] == "linear":
        return freq / how["factor"], 1.0
    turns = how["original"] * freq / (2 * math.pi)          # turns of the pair over the original context
    if how["kind"] == "bands":                              # from 1 to 4 turns: between stretched and as it was
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        return freq / how["factor"] * (1 - keep) + freq * keep, 1.0
    edge = lambda r: dims * math.log(how["original"] / (2 * math.pi * r)) / (2 * math.log(base))
    lo, hi = max(0, math.floor(edge(32.0))), min(dims - 1, math.ceil(edge(1.0)))
    keep = 1.0 - ((i - lo) / max(0.001, hi - lo)).clamp(0.0, 1.0)
    return freq / how["factor"] * (1 - keep) + freq * keep, 0.1 * math.log(how["factor"]) + 1.0


def _turned(x, weight, angles, amplitude, case):
    """Norm and rotation of x [n][H][rows][d] (32 or 64 bits), angles [n][rows][dims / 2]."""
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
    c, s = ((f(angles) * amplitude).to(x.dtype)[:, None] for f in (torch.cos, torch.sin))
    dims = case["dims"]
    if case["layout"] == "half":
        a, b = x[..., :dims // 2], x[..., dims // 2:dims]
        return torch.cat((a * c - b * s, b * c + a * s, x[..., dims:]), -1)
    a, b = x[..., 0:dims:2], x[..., 1:dims:2]
    return torch.cat((torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2), x[..., dims:]), -1)


def _angles(s, rows):
    freq, amplitude = _frequencies(s.case)
    p = s.positions[:, None].double() + torch.arange(rows, device="cuda")
    return p[..., None] * freq, amplitude


def _rotate(s):
    if own:
        s.rotary.apply(s.q, s.k, s.q_out, s.k_out, positions=s.positions, lengths=s.lengths)
        return s.q_out, s.k_out
    n = s.case["n"]
    angles, amplitude = _angles(s, n)
    live = (torch.arange(n, device="cuda") < s.lengths[:, None])[:, None, :, None]
    for x, w, out in ((s.q, s.qw, s.q_out), (s.k, s.kw, s.k_out)):
        out.copy_(torch.where(live, _turned(x.float(), w, angles, amplitude, s.case).bfloat16(), out))
    return s.q_out, s.k_out


def _store(s):
    c = s.case
    if own:
        s.cache.store_rotated(0, s.rotary, s.q, s.src_k, s.src_v, s.q_out, positions=s.positions, counts=s.new)
        return dict(q=s.q_out, k=s.k, v=s.v, k_scale=s.k_scale, v_scale=s.v_scale)
    page, rows = c["page"], c["rows"]
    angles, amplitude = _angles(s, rows)
    live = (torch.arange(rows, device="cuda") < s.new[:, None])[:, None, :, None]
    s.q_out.copy_(torch.where(live, _turned(s.q.float(), s.qw, angles, amplitude, c).bfloat16(), s.q_out))
    key = _turned(s.src_k.float(), s.kw, angles, amplitude, c).bfloat16()       # as the rotation alone would leave them
    start = (s.length - s.new).long()
    cols = (start // page)[:, None] + torch.arange((rows + page - 2) // page + 1, device="cuda")  # touched pages
    touched = (cols < s.count[:, None]) & (s.new > 0)[:, None]
    seq, col = touched.nonzero(as_tuple=True)
    pg = s.table[seq, cols[seq, col]].long()
    pos = cols[seq, col][:, None] * page + torch.arange(page, device="cuda")
    row = pos - start[seq][:, None]
    new = (row >= 0) & (row < s.new[seq][:, None])
    old = row < 0
    for src, codes, scales in ((key, s.k, s.k_scale), (s.src_v, s.v, s.v_scale)):
        x = src.transpose(1, 2)[seq[:, None], row.clamp(0, rows - 1)].float().transpose(1, 2)   # [pages][H][page][d]
        fresh = _page_scale(torch.where(new[:, None, :, None], x.abs(), torch.zeros((), device="cuda")).amax((2, 3)),
                            s.code)
        held = scales[0][pg]
        scale = torch.where(old.any(-1)[:, None], torch.maximum(held, fresh), fresh)
        was = codes[0].view(torch.uint8)[pg].view(codes.dtype)
        again = _encode(was.float() * held[..., None, None] / scale[..., None, None], s.code)
        put = _encode(x / scale[..., None, None], s.code)
        keep = torch.where(old[:, None, :, None], again.view(torch.uint8), was.view(torch.uint8))
        codes[0].view(torch.uint8)[pg] = torch.where(new[:, None, :, None], put.view(torch.uint8), keep)
        scales[0][pg] = scale
    return dict(q=s.q_out, k=s.k, v=s.v, k_scale=s.k_scale, v_scale=s.v_scale)


def _read(s):
    if own:
        s.cache.read(0, s.k_out, s.v_out, starts=s.starts, counts=s.counts)
        return s.k_out, s.v_out
    page, rows = s.case["page"], s.k_out.shape[2]
    row = torch.arange(rows, device="cuda")
    tok = torch.minimum(s.starts[:, None] + row, (s.length - 1).clamp_min(0)[:, None]).long()    # [n][rows]
    live = (row < s.counts[:, None])[:, None, :, None]
    pg = s.table.gather(1, tok // page).clamp_min(0).long()[:, None]
    head = torch.arange(s.case["Hkv"], device="cuda")[:, None]
    for codes, scales, out in ((s.k, s.k_scale, s.k_out), (s.v, s.v_scale, s.v_out)):
        raw = codes[0].view(torch.uint8)[pg, head, (tok % page)[:, None]].view(codes.dtype)      # [n][H][rows][d]
        out.copy_(torch.where(live, (raw.float() * scales[0][pg, head][..., None]).bfloat16(), out))
    return s.k_out, s.v_out


def _attention(s):
    c = s.case
    if own:
        s.cache.shared_attention(0, s.q, s.out, s.groups)
        return s.out
    n, Hq, H, T, d = len(s.length), c["Hq"], c["Hkv"], c["T"], c["d"]
    pages = s.table.clamp_min(0).long()
    k, v = ((codes[0].view(torch.uint8)[pages].view(codes.dtype).float() * scale[0][pages][..., None, None])
            .transpose(1, 2).reshape(n, H, -1, d) for codes, scale in ((s.k, s.k_scale), (s.v, s.v_scale)))
    j = torch.arange(k.shape[2], device="cuda")
    i = s.length[:, None].long() - T + torch.arange(T, device="cuda")                     # [n][T]
    v = torch.where((j < s.length[:, None])[:, None, :, None], v, torch.zeros((), device="cuda"))
    x = s.q.float().reshape(n, H, Hq // H * T, d) @ k.transpose(-1, -2) / math.sqrt(d)
    seen = (j <= i[..., None])[:, None, None]
    x = x.reshape(n, H, Hq // H, T, -1).masked_fill(~seen, -math.inf).reshape(n, H, Hq // H * T, -1)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    o = torch.where(total > 0, p @ v / total, torch.zeros((), device="cuda"))
    s.out.copy_(o.reshape(n, Hq, T, d))
    return s.out


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_scale(amax):
    """The e4m3 page scale from the largest magnitude, a Python float (0: an empty page)."""
    return max(2.0 ** math.ceil(math.log2(amax / 448.0)), SCALE_MIN) if amax > 0 else SCALE_MIN


def _exact_e4m3(x):
    """The nearest e4m3 value (ties to even), |x| <= 448, in float64."""
    e = torch.floor(torch.log2(x.abs().clamp_min(1e-300))).clamp_min(-6.0)
    step = torch.exp2(e - 3.0)
    return torch.round(x / step) * step


def _exact_turned(x, weight, first, case):
    """Rows of one sequence [H][rows][d], the first at position `first`: complex numbers, a pair each."""
    x, dims = x.double(), case["dims"]
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["d"] + EPS) * weight.double()
    freq, amplitude = _frequencies(case)
    angle = torch.arange(first, first + x.shape[1], dtype=torch.float64, device="cuda")[:, None] * freq
    turn = torch.polar(torch.full_like(angle, amplitude), angle)
    y = x.clone()
    at = (slice(0, dims // 2), slice(dims // 2, dims)) if case["layout"] == "half" else (slice(0, dims, 2), slice(1, dims, 2))
    z = torch.complex(x[..., at[0]].contiguous(), x[..., at[1]].contiguous()) * turn
    y[..., at[0]], y[..., at[1]] = z.real, z.imag
    return y


def exact(case, seed):
    op = case["op"]
    global own
    mine, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = mine
    if op == "rotate":
        res = []
        for x, w in ((s.q, s.qw), (s.k, s.kw)):
            out = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
            for b, (n, first) in enumerate(zip(s.lengths.tolist(), s.positions.tolist())):
                out[b, :, :n] = _exact_turned(x[b, :, :n], w, first, case)
            res.append(out)
        return tuple(res)
    if op == "store":
        old, new = _stored(case)
        page = case["page"]
        if sum(-(-x // page) + 1 for x in new) * case["Hkv"] > 30000:
            return None
        res = dict(q=torch.zeros(s.q.shape, dtype=torch.float64, device="cuda"))
        for name, codes, scales in (("k", s.k, s.k_scale), ("v", s.v, s.v_scale)):
            codes, scales = codes.double(), scales.double()
            for b, (o, c, first) in enumerate(zip(old, new, s.positions.tolist())):
                if name == "k":
                    res["q"][b, :, :c] = _exact_turned(s.q[b, :, :c], s.qw, first, case)
                    rows = _exact_turned(s.src_k[b, :, :c], s.kw, first, case).bfloat16().double()
                else:
                    rows = s.src_v[b, :, :c].double()
                table = s.table[b].tolist()
                for col in range(o // page, -(-(o + c) // page) if c else 0):
                    pg = table[col]
                    a, z = max(o, col * page), min(o + c, (col + 1) * page)        # new positions of this page
                    x = rows[:, a - o:z - o]
                    top, held = x.abs().amax((1, 2)).tolist(), scales[0, pg].tolist()
                    sc = torch.tensor([max(_exact_scale(t), w if a > col * page else 0.0) for t, w in zip(top, held)],
                                      dtype=torch.float64, device="cuda")
                    before = codes[0, pg, :, :a - col * page] * (scales[0, pg] / sc)[:, None, None]
                    codes[0, pg, :, :a - col * page] = _exact_e4m3(before)
                    codes[0, pg, :, a - col * page:z - col * page] = _exact_e4m3(x / sc[:, None, None])
                    scales[0, pg] = sc
            res[name] = codes
            res[name + "_scale"] = scales
        return res
    if op == "read":
        page, res = case["page"], []
        for codes, scales, out in ((s.k, s.k_scale, s.k_out), (s.v, s.v_scale, s.v_out)):
            out = out.double()
            for b, (a, c) in enumerate(zip(*_newest(case))):
                pages = s.table[b, a // page:-(-(a + c) // page)].long()
                x = codes[0].view(torch.uint8)[pages].view(codes.dtype).double() * scales[0][pages].double()[..., None, None]
                x = x.transpose(0, 1).reshape(case["Hkv"], -1, case["d"])
                out[b, :, :c] = x[:, a % page:a % page + c]
            res.append(out)
        return tuple(res)
    n, Hq, H, T, d, page = len(s.length), case["Hq"], case["Hkv"], case["T"], case["d"], case["page"]
    out = torch.zeros(n, Hq, T, d, dtype=torch.float64, device="cuda")
    for b, L in enumerate(s.length.tolist()):
        pages = s.table[b, :-(-L // page)].long()
        k, v = ((c[0].view(torch.uint8)[pages].view(c.dtype).double() * sc[0][pages].double()[..., None, None])
                .transpose(0, 1).reshape(H, -1, d)[:, :L] for c, sc in ((s.k, s.k_scale), (s.v, s.v_scale)))
        for t in range(T):
            i = L - T + t
            if i >= 0:
                q = s.q[b, :, t].double().reshape(H, Hq // H, d)
                x = q @ k[:, :i + 1].transpose(-1, -2) / math.sqrt(d)
                out[b, :, t] = (torch.softmax(x, -1) @ v[:, :i + 1]).reshape(Hq, d)
    return out
