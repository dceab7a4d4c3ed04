"""What is measured of the batched serving operators: appending to a paged
KV cache, attention of single tokens over it, and matrix-vector products with
4-bit weights.

``run`` computes each operator in its plain form (elementary torch operations
in 32 bits, rounded once at the end) or, where ``own`` is true, by the calls a
user makes of the package.  ``exact`` gives the operators' definitions in 64
bits, written apart from the plain form.

Shapes: the decoder heads 16:8 of 128 and the widths 1024, 2048 and 6144 are
the framework's 0.6B and 1.7B shapes, 8:2 heads of 64 its grouped-query test
shape, the position sections 24, 20, 20 its talker's.
"""
import math
import random

import torch

own = False

THETA = 1e6
EPS = 1e-6
E4M3 = torch.float8_e4m3fn
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "e4m3": E4M3}
SIZE = {"fp32": 4, "bf16": 2, "e4m3": 1}


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one new audio token of the talker: its key and value rotated by three position streams
        dict(name="append_one", op="append", rows=1, pad=0, prompts=0, lo=300, hi=300, seed=0, hq=16, hkv=8, d=128,
             x="fp32", cache="bf16", page=16, norm=True, streams=1),
        # a decode step of a full batch, captured for 256 rows of which 250 are in use
        dict(name="append_batch", op="append", rows=256, pad=6, prompts=0, lo=16, hi=8000, seed=1, hq=16, hkv=8, d=128,
             x="bf16", cache="bf16", page=16, norm=True, streams=0),
        # several prompts' keys and values at once into an 8-bit cache, pages of an odd size
        dict(name="append_prompts", op="append", rows=20011, pad=0, prompts=5, lo=0, hi=0, seed=2, hq=16, hkv=8, d=128,
             x="bf16", cache="e4m3", page=24, norm=True, streams=0),
        # one sequence early in its decode, the framework's own fp32 activations
        dict(name="attend_one", op="attend", rows=1, lo=257, hi=257, seed=0, hq=16, hkv=8, d=128, x="fp32", cache="bf16",
             page=16, window=0),
        # the same sequence at the end of the long-context workload
        dict(name="attend_long", op="attend", rows=1, lo=5119, hi=5119, seed=0, hq=16, hkv=8, d=128, x="fp32", cache="bf16",
             page=16, window=0),
        # a serving batch: lengths from a first token to thousands, a row without tokens among them
        dict(name="attend_ragged", op="attend", rows=64, lo=0, hi=8192, seed=3, hq=16, hkv=8, d=128, x="bf16", cache="bf16",
             page=16, window=0),
        # many short sequences, 64-wide heads, odd pages, a sliding window
        dict(name="attend_many_short", op="attend", rows=256, lo=1, hi=500, seed=4, hq=8, hkv=2, d=64, x="bf16",
             cache="bf16", page=24, window=300),
        # a batch of long contexts in an 8-bit cache
        dict(name="attend_fp8_long", op="attend", rows=16, lo=30001, hi=32768, seed=5, hq=16, hkv=8, d=128, x="bf16",
             cache="e4m3", page=64, window=0),
        # the stacked q/k/v projection of the 0.6B shape for one token
        dict(name="matvec_qkv", op="matvec", m=1, n=4096, k=1024, x="fp32", group=64, zeros=False, residual=False),
        # its head over the whole vocabulary
        dict(name="matvec_head", op="matvec", m=1, n=151936, k=1024, x="fp32", group=128, zeros=False, residual=False),
        # gate and up of the 1.7B shape for eight sequences, small groups with zero points
        dict(name="matvec_gate_up", op="matvec", m=8, n=12288, k=2048, x="bf16", group=32, zeros=True, residual=False),
        # its down projection for three sequences, added to the residual stream
        dict(name="matvec_down", op="matvec", m=3, n=2048, k=6144, x="fp32", group=64, zeros=False, residual=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "matvec"])
    if op == "matvec":
        m = rng.randint(1, 16)
        k = 128 * _log_int(rng, 2, 64)
        n = _log_int(rng, 64, min(151936, 400_000_000 // k))
        group = rng.choice([32, 64, 128])
        return dict(op=op, m=m, n=n, k=k, x=rng.choice(["fp32", "bf16"]), group=group, zeros=rng.random() < 0.5,
                    residual=rng.random() < 0.5)
    hkv, g, d = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 6, 8, 16]), rng.choice([64, 128])
    c = dict(op=op, hq=hkv * g, hkv=hkv, d=d, x=rng.choice(["fp32", "bf16"]), cache=rng.choice(["bf16", "e4m3"]),
             page=rng.choice([8, 16, 16, 24, 32, 64, 100, 128]), seed=rng.randrange(1 << 20))
    if op == "append":
        prompts = rng.choice([0, 0, 1, 4])
        rows = _log_int(rng, 1, 512) if not prompts else _log_int(rng, 16, 20000)
        return dict(c, rows=rows, prompts=prompts, pad=0 if prompts else rng.randint(0, rows // 8), lo=1, hi=_log_int(rng, 2, 4096),
                    norm=rng.random() < 0.5, streams=rng.choice([0, 0, 1, 2]))
    rows = _log_int(rng, 1, 256)
    hi = _log_int(rng, 4, max(4, min(65536, 60_000_000 // (rows * hkv * d))))
    return dict(c, rows=rows, lo=rng.choice([0, 1, hi // 2, hi]), hi=hi, window=rng.choice([0, 0, 0, max(1, hi // 3)]))


def _lengths(case):
    """Tokens of each sequence, from the case alone: spread over the logarithm of its range."""
    rng = random.Random(case["seed"])
    lo, hi = case["lo"], case["hi"]
    n = [lo if lo == hi else int(round(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 1))))) - 1
         for _ in range(case["rows"])]
    if lo < hi and case["rows"] > 1:
        n[rng.randrange(case["rows"])] = lo
    return n


def _appended(case):
    """(sequence, slot) of each row of an append; the rows of a padded batch's end have slot -1."""
    if case["prompts"]:
        rng = random.Random(case["seed"])
        cuts = sorted(rng.sample(range(1, case["rows"]), min(case["prompts"], case["rows"]) - 1)) if case["prompts"] > 1 else []
        ends = cuts + [case["rows"]]
        seqs, slots, at = [], [], 0
        for i, e in enumerate(ends):
            seqs += [i] * (e - at)
            slots += list(range(e - at))
            at = e
        return seqs, slots
    slots = _lengths(case)
    for i in range(case["rows"] - case["pad"], case["rows"]):
        slots[i] = -1
    return list(range(case["rows"])), slots


def _streams(case):
    """Rotary pairs that each of three position streams drives, or None for one position a token."""
    half = case["d"] // 2
    return (half - 2 * (5 * half // 16), 5 * half // 16, 5 * half // 16) if case["streams"] else None


# ---------------------------------------------------------------------------
# the inputs
# ---------------------------------------------------------------------------

def _pages(counts, page, g, dev):
    """A page table for sequences of ``counts`` tokens, its pages in random order, and the number of pages."""
    need = torch.tensor([-(-c // page) for c in counts])
    total = int(need.sum()) + 3
    width = max(1, int(need.max()))
    order = torch.randperm(total, generator=g, device=dev).int()
    first = (need.cumsum(0) - need).to(dev)
    col = torch.arange(width, device=dev)
    at = (first[:, None] + col).clamp_max(total - 1)
    used = col < need.to(dev)[:, None]
    return torch.where(used, order[at], torch.full_like(order[at], -1)), total


def _normal(shape, g, dev, dtype, gain=1.0):
    return (torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16 if dtype == E4M3 else dtype) * gain).to(dtype)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    x = TYPES[case["x"]]
    if case["op"] == "matvec":
        m, n, k, group = case["m"], case["n"], case["k"], case["group"]
        s = dict(x=_normal((m, k), g, dev, x),
                 codes=torch.randint(0, 256, (n, k // 2), generator=g, device=dev, dtype=torch.uint8),
                 scales=((torch.rand((n, k // group), generator=g, device=dev) + 0.5) * 0.006).bfloat16(), zeros=None, residual=None)
        if case["zeros"]:
            s["zeros"] = torch.randint(4, 12, (n, k // group), generator=g, device=dev, dtype=torch.uint8)
        if case["residual"]:
            s["residual"] = _normal((m, n), g, dev, x)
        return dict(s, case=case)
    hq, hkv, d, page, cache = case["hq"], case["hkv"], case["d"], case["page"], TYPES[case["cache"]]
    s = dict(case=case, k_scale=None, v_scale=None)
    if cache == E4M3:
        s["k_scale"] = torch.rand(hkv, generator=g, device=dev) * 0.02 + 0.01
        s["v_scale"] = torch.rand(hkv, generator=g, device=dev) * 0.02 + 0.01
    fill = 1.0 if cache != E4M3 else 48.0    # a cache of 8 bits holds values / scale
    if case["op"] == "append":
        seqs, slots = _appended(case)
        counts = [0] * (max(seqs) + 1)
        for q, p in zip(seqs, slots):
            counts[q] = max(counts[q], p + 1)
        s["table"], total = _pages(counts, page, g, dev)
        for c in ("k_cache", "v_cache"):
            s[c] = _normal((total, hkv, page, d), g, dev, cache, fill)
        # one projection's output holds the three: rows of q, k and v heads
        qkv = _normal((case["rows"], hq + 2 * hkv, d), g, dev, x)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["q_out"] = torch.zeros((case["rows"], hq, d), device=dev, dtype=x)
        s["seqs"] = torch.tensor(seqs, device=dev, dtype=torch.int32) if case["prompts"] else None
        s["slots"] = torch.tensor(slots, device=dev, dtype=torch.int32)
        s["sections"] = _streams(case)
        p = s["slots"]
        s["positions"] = torch.stack([p, p + 7, 2 * p + 3]).clamp_min(0).contiguous() if s["sections"] else None
        rows = 2 * max(slots) + 8
        half = d // 2
        w = THETA ** (-torch.arange(half, device=dev, dtype=torch.float64) * 2 / d)
        a = torch.arange(rows, device=dev, dtype=torch.float64)[:, None] * w
        s["rope"] = torch.stack([a.cos(), a.sin()], -1).float().contiguous()
        s["q_norm"] = s["k_norm"] = None
        if case["norm"]:
            s["q_norm"] = (1 + 0.02 * torch.randn(d, generator=g, device=dev)).bfloat16()
            s["k_norm"] = (1 + 0.02 * torch.randn(d, generator=g, device=dev)).bfloat16()
        return s
    lengths = _lengths(case)
    s["table"], total = _pages(lengths, page, g, dev)
    for c in ("k_cache", "v_cache"):
        s[c] = _normal((total, hkv, page, d), g, dev, cache, fill)
    s["lengths"] = torch.tensor(lengths, device=dev, dtype=torch.int32)
    # what earlier tenants of the last pages left behind the last token is no number
    last = s["table"].gather(1, ((s["lengths"].long() - 1).clamp_min(0) // page)[:, None])[:, 0]
    some = (s["lengths"] % page > 0).nonzero()[:, 0]
    for c in ("k_cache", "v_cache"):
        rows = s[c].view(torch.uint8 if cache == E4M3 else cache)
        tail = torch.arange(page, device=dev) >= (s["lengths"] % page)[some, None]
        at = last[some].long()[:, None].expand_as(tail)[tail], torch.arange(page, device=dev).expand_as(tail)[tail]
        rows[at[0], :, at[1]] = 0x7F if cache == E4M3 else float("nan")
    s["q"] = _normal((case["rows"], hq, d), g, dev, x, 2.0)
    s["window"] = case["window"]
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return {"append": _append, "attend": _attend, "matvec": _matvec}[s["case"]["op"]](s)


def _mk():
    import persistent_transformer_megakernel_gb300 as mk
    return mk


def _stored(x, cache, scale):
    """Values as a cache holds them: [rows][heads][d] fp32 over the head's scale, rounded."""
    if scale is not None:
        x = (x / scale[:, None]).clamp(-448.0, 448.0)
    return x.to(cache.dtype)


def _rotated(x, gain, cos, sin):
    x = x.float()
    if gain is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain.float()
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _append(s):
    if own:
        q = _mk().paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["slots"], seqs=s["seqs"], q=s["q"],
                               q_out=s["q_out"], rope=s["rope"], positions=s["positions"], mrope_sections=s["sections"],
                               mrope_interleaved=s["case"]["streams"] == 2, q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS,
                               k_scale=s["k_scale"], v_scale=s["v_scale"])
        return [q, s["k_cache"], s["v_cache"]]
    page = s["k_cache"].shape[2]
    live = (s["slots"] >= 0).nonzero()[:, 0]
    slot = s["slots"][live].long()
    seq = live if s["seqs"] is None else s["seqs"][live].long()
    half = s["k"].shape[2] // 2
    if s["sections"] is None:
        cs = s["rope"][slot]
    else:
        i = torch.arange(half, device=slot.device)
        n0, n1, n2 = s["sections"]
        if s["case"]["streams"] == 1:
            stream = (i >= n0).long() + (i >= n0 + n1).long()
        else:
            stream = torch.where((i % 3 == 1) & (i < 3 * n1), 1, torch.where((i % 3 == 2) & (i < 3 * n2), 2, 0))
        at = s["positions"][:, live].long()[stream]                 # [half][rows]
        cs = s["rope"][at.t(), i]
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
    s["q_out"][live] = _rotated(s["q"][live], s["q_norm"], cos, sin).to(s["q"].dtype)
    at = s["table"][seq, slot // page].long(), slot % page
    s["k_cache"][at[0], :, at[1]] = _stored(_rotated(s["k"][live], s["k_norm"], cos, sin), s["k_cache"], s["k_scale"])
    s["v_cache"][at[0], :, at[1]] = _stored(s["v"][live].float(), s["v_cache"], s["v_scale"])
    return [s["q_out"], s["k_cache"], s["v_cache"]]


def _attend(s):
    q = s["q"]
    if own:
        lse = torch.empty(q.shape[:2], device=q.device, dtype=torch.float32)
        out = _mk().paged_attention(q, s["k_cache"], s["v_cache"], s["table"], s["lengths"], window=s["window"],
                                    k_scale=s["k_scale"], v_scale=s["v_scale"], lse=lse)
        return [out, lse]
    rows, hq, d = q.shape
    hkv, page = s["k_cache"].shape[1:3]
    pos = torch.arange(s["table"].shape[1] * page, device=q.device)
    there = pos < s["lengths"][:, None]
    if s["window"]:
        there &= pos >= s["lengths"][:, None] - s["window"]
    at = s["table"].clamp_min(0).long()[:, pos // page], pos % page
    k = s["k_cache"][at[0], :, at[1]].float()                       # [rows][positions][hkv][d]
    v = s["v_cache"][at[0], :, at[1]].float()
    v.masked_fill_(~there[:, :, None, None], 0.0)
    if s["k_scale"] is not None:
        k *= s["k_scale"][:, None]
        v *= s["v_scale"][:, None]
    qs = q.float().view(rows, hkv, hq // hkv, d) * d ** -0.5
    z = torch.matmul(qs, k.permute(0, 2, 3, 1))                     # [rows][hkv][group][positions]
    z.masked_fill_(~there[:, None, None, :], -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, 1.0)
    lse = torch.log(total) + torch.where(torch.isinf(top), 0.0, top)
    return [out.view(rows, hq, d).to(q.dtype), lse.view(rows, hq)]


def _matvec(s):
    x, codes, scales = s["x"], s["codes"], s["scales"]
    if own:
        return _mk().matvec_q4(x, codes, scales, zeros=s["zeros"], residual=s["residual"])
    n, k = codes.shape[0], 2 * codes.shape[1]
    w = torch.stack([codes & 15, codes >> 4], -1).view(n, scales.shape[1], -1).float()
    w = (w - (8.0 if s["zeros"] is None else s["zeros"].float()[..., None])) * scales.float()[..., None]
    y = torch.matmul(x.float(), w.view(n, k).t())
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(x.dtype)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    xs = SIZE[case["x"]]
    if case["op"] == "matvec":
        m, n, k = case["m"], case["n"], case["k"]
        b = n * k // 2 + n * (k // case["group"]) * (3 if case["zeros"] else 2) + m * k * xs
        return dict(bytes=b + m * n * xs * (2 if case["residual"] else 1), flops=2 * m * n * k)
    hq, hkv, d, cs = case["hq"], case["hkv"], case["d"], SIZE[case["cache"]]
    if case["op"] == "append":
        slots = [p for p in _appended(case)[1] if p >= 0]
        row = (2 * hq + 2 * hkv) * d * xs + 2 * hkv * d * cs
        return dict(bytes=len(slots) * (row + 8) + len(set(slots)) * d * 4, flops=len(slots) * (hq + hkv) * d * (10 if case["norm"] else 6))
    lengths = [min(n, case["window"]) if case["window"] else n for n in _lengths(case)]
    tokens = sum(lengths)
    b = tokens * hkv * d * 2 * cs + case["rows"] * hq * (2 * d * xs + 4) + 4 * sum(-(-n // case["page"]) for n in lengths)
    return dict(bytes=b, flops=4 * tokens * hq * d)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "matvec": _exact_matvec}[case["op"]](case, s)


def _exact_append(case, s):
    f = torch.float64
    d, page = case["d"], case["page"]
    half = d // 2
    seqs, slots = _appended(case)
    rows = [r for r, p in enumerate(slots) if p >= 0]
    if not rows:
        return [s["q_out"].to(f), s["k_cache"].to(f), s["v_cache"].to(f)]
    dev = s["k"].device
    r = torch.tensor(rows, device=dev)
    p = torch.tensor([slots[i] for i in rows], device=dev)
    u = torch.tensor([seqs[i] for i in rows], device=dev)
    angle = torch.empty((len(rows), half), device=dev, dtype=f)
    for i in range(half):
        at = p.to(f)
        if case["streams"]:
            n0, n1, n2 = _streams(case)
            if case["streams"] == 1:
                which = 0 if i < n0 else 1 if i < n0 + n1 else 2
            else:
                which = i % 3 if i % 3 and i < 3 * (n1 if i % 3 == 1 else n2) else 0
            at = (at, at + 7, 2 * at + 3)[which]
        angle[:, i] = at * THETA ** (-2 * i / d)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def turned(x, gain):
        x = x[r].to(f)
        if gain is not None:
            x = gain.to(f) * x / ((x ** 2).sum(-1, keepdim=True) / d + EPS).sqrt()
        z = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * turn
        return torch.cat([z.real, z.imag], -1)

    q = s["q_out"].to(f)
    q[r] = turned(s["q"], s["q_norm"])
    to = s["table"][u, p // page].long()
    out = [q]
    for c, x, scale in (("k_cache", turned(s["k"], s["k_norm"]), s["k_scale"]), ("v_cache", s["v"][r].to(f), s["v_scale"])):
        held = s[c].to(f)
        if scale is not None:
            x = (x / scale.to(f)[None, :, None]).clamp(-448, 448)
        held[to, :, p % page] = x
        out.append(held)
    return out


def _exact_attend(case, s):
    f = torch.float64
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    out = torch.zeros((case["rows"], hq, d), device=s["q"].device, dtype=f)
    lse = torch.full((case["rows"], hq), -math.inf, device=s["q"].device, dtype=f)
    for b, n in enumerate(_lengths(case)):
        first = max(0, n - case["window"]) if case["window"] else 0
        if n == first:
            continue
        pages = s["table"][b, : -(-n // page)].long()
        held = []
        for c, scale in (("k_cache", s["k_scale"]), ("v_cache", s["v_scale"])):
            x = s[c][pages].transpose(0, 1).reshape(hkv, -1, d)[:, first:n].to(f)
            held.append(x if scale is None else x * scale.to(f)[:, None, None])
        q = s["q"][b].to(f).view(hkv, hq // hkv, d)
        z = torch.einsum("hgd,hnd->hgn", q, held[0]) / math.sqrt(d)
        out[b] = torch.einsum("hgn,hnd->hgd", z.softmax(-1), held[1]).reshape(hq, d)
        lse[b] = z.logsumexp(-1).reshape(hq)
    return [out, lse]


def _exact_matvec(case, s):
    f = torch.float64
    m, n, k, group = case["m"], case["n"], case["k"], case["group"]
    y = torch.zeros((m, n), device=s["x"].device, dtype=f) if s["residual"] is None else s["residual"].to(f)
    x = s["x"].to(f)
    step = max(1, (1 << 26) // k)
    for a in range(0, n, step):
        c = s["codes"][a:a + step].to(torch.int32)
        w = torch.empty((c.shape[0], k), device=c.device, dtype=f)
        w[:, 0::2], w[:, 1::2] = (c % 16).to(f), (c // 16).to(f)
        z = 8.0 if s["zeros"] is None else s["zeros"][a:a + step].to(f).repeat_interleave(group, 1)
        y[:, a:a + step] += x @ ((w - z) * s["scales"][a:a + step].to(f).repeat_interleave(group, 1)).t()
    return y
