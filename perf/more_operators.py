"""What is measured of the operators that take several sequences' prompts through
the batched path: page tables and slot maps from request lengths, attention with
a sliding window and first tokens that stay visible (whole prompts and single
tokens), products in 8-bit floating point with block scales, and the adjustment
of logits before a token is chosen.

``run`` computes each operator in its plain form (elementary torch operations
in 32 bits, rounded once at the end) or, where ``own`` is true, by the calls a
user makes of the package.  ``exact`` gives the operators' definitions in 64
bits, written apart from the plain form.

Shapes: the decoder heads 16:8 of 128 and the widths 1024, 2048, 6144 and 151936
are the framework's 0.6B and 1.7B shapes, 8:2 heads of 64 its grouped-query test
shape.
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "e4m3": E4M3}
SIZE = {"fp32": 4, "bf16": 2, "e4m3": 1}
BLOCK = 128


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a decode step's bookkeeping: 64 sequences get a token each, some of them a new page, two rows are padding
        dict(name="plan_step", op="plan", n=64, pad=2, lo=16, hi=8000, step=True, hi_new=1, rows=64, page=16, short=False, seed=0),
        # the same for a mixed batch: whole and continued prompts of up to thousands of tokens among decoding sequences
        dict(name="plan_prompts", op="plan", n=512, pad=5, lo=0, hi=16000, step=False, hi_new=6000, rows=131072, page=16, short=False,
             seed=1),
        # a decode step of one long sequence that sees its last 1024 tokens and the first four, fp32 activations
        dict(name="sinks_one", op="token", rows=1, lo=5119, hi=5119, hq=16, hkv=8, d=128, x="fp32", cache="bf16", page=16, window=1024,
             sinks=4, seed=2),
        # a decode batch of long sequences under a window of 4096, 8-bit cache
        dict(name="sinks_batch", op="token", rows=96, lo=100, hi=30000, hq=16, hkv=8, d=128, x="bf16", cache="e4m3", page=64,
             window=4096, sinks=16, seed=3),
        # one short prompt: latency
        dict(name="prompt_short", op="prompt", n=1, lo_new=77, hi_new=77, lo_old=0, hi_old=0, hq=16, hkv=8, d=128, cache="bf16",
             page=16, window=0, sinks=0, seed=4),
        # one long prompt, causal
        dict(name="prompt_long", op="prompt", n=1, lo_new=8192, hi_new=8192, lo_old=0, hi_old=0, hq=16, hkv=8, d=128, cache="bf16",
             page=16, window=0, sinks=0, seed=5),
        # a batch of prompts' chunks behind what is cached, window and first tokens, 64-wide heads of 4 to a key head, 8 bits
        dict(name="prompt_chunks", op="prompt", n=13, lo_new=1, hi_new=2500, lo_old=0, hi_old=9000, hq=8, hkv=2, d=64, cache="e4m3",
             page=24, window=1500, sinks=4, seed=6),
        # the stacked q/k/v projection of the 0.6B shape for a decode batch
        dict(name="fp8_step", op="product", m=8, n=4096, k=1024, x="bf16", out="bf16", residual=False),
        # the down projection of the 1.7B shape for a ragged batch of prompts, added to the residual stream
        dict(name="fp8_down", op="product", m=777, n=2048, k=6144, x="bf16", out="fp32", residual=True),
        # gate and up of the 1.7B shape for long prompts
        dict(name="fp8_gate_up", op="product", m=8192, n=12288, k=2048, x="bf16", out="bf16", residual=False),
        # one sequence's logits under a grammar's mask, with its history's penalties
        dict(name="logits_one", op="logits", n=1, vocab=151936, x="fp32", history=700, penalties=True, biases=0, mask=True, seed=7),
        # a batch's logits: long histories, a few biased tokens each, a mask
        dict(name="logits_batch", op="logits", n=64, vocab=151936, x="bf16", history=6000, penalties=True, biases=40, mask=True, seed=8),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "token", "prompt", "prompt", "product", "product", "logits"])
    seed = rng.randrange(1 << 20)
    if op == "plan":
        n, step = _log_int(rng, 1, 512), rng.random() < 0.4
        hi_new = 1 if step else _log_int(rng, 1, 6000)
        return dict(op=op, n=n, pad=rng.randint(0, n // 8), lo=0, hi=_log_int(rng, 2, 16000), step=step, hi_new=hi_new,
                    rows=n if step else min(131072, n * hi_new + rng.randint(0, 100)), page=rng.choice([1, 8, 16, 16, 24, 32, 64, 100]),
                    short=rng.random() < 0.15, seed=seed)
    if op == "logits":
        n = _log_int(rng, 1, 64)
        return dict(op=op, n=n, vocab=_log_int(rng, 200, 151936), x=rng.choice(["fp32", "bf16"]) if n <= 32 else "bf16",
                    history=rng.choice([0, _log_int(rng, 1, 6000)]), penalties=rng.random() < 0.7, biases=rng.choice([0, 1, 40, 300]),
                    mask=rng.random() < 0.6, seed=seed)
    if op == "product":
        m, k = _log_int(rng, 1, 8192), 16 * _log_int(rng, 8, 512)
        n = _log_int(rng, 64, max(64, min(151936, 200_000_000_000 // (m * k))))
        return dict(op=op, m=m, n=n, k=k, x=rng.choice(["fp32", "bf16"]), out=rng.choice(["fp32", "bf16"]), residual=rng.random() < 0.4)
    hkv, g, d = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 6, 8, 16]), rng.choice([64, 128])
    c = dict(op=op, hq=hkv * g, hkv=hkv, d=d, cache=rng.choice(["bf16", "e4m3"]), page=rng.choice([8, 16, 16, 24, 32, 64, 100, 128]), seed=seed,
             sinks=rng.choice([0, 1, 4, 16, 130]))
    if op == "token":
        rows, window = _log_int(rng, 1, 128), _log_int(rng, 1, 4096)
        hi = _log_int(rng, 4, max(4, min(65536, 60_000_000 // (rows * hkv * d))))
        return dict(c, rows=rows, lo=rng.choice([0, 1, hi // 2, hi]), hi=hi, x=rng.choice(["fp32", "bf16"]), window=window)
    n = _log_int(rng, 1, 24)
    old = rng.choice([0, _log_int(rng, 1, 12000)])
    new = _log_int(rng, 1, max(1, min(6000, 60_000_000 // (n * c["hq"] * (old + 3000)))))
    return dict(c, n=n, lo_new=rng.choice([0, 1, new]), hi_new=new, lo_old=rng.choice([0, old]), hi_old=old,
                window=rng.choice([0, 0, _log_int(rng, 1, 4096)]))


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over the logarithm."""
    return lo if lo == hi else max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 1))))) - 1))


def _planned(case):
    """Tokens that each sequence has (-1: a padding row) and gets."""
    rng = random.Random(case["seed"])
    n, left = case["n"], case["rows"]
    lengths, counts = [], []
    for i in range(n):
        pad = i >= n - case["pad"]
        lengths.append(-1 if pad else _spread(rng, case["lo"], case["hi"]))
        c = 1 if case["step"] or rng.random() < 0.6 else _spread(rng, 0, case["hi_new"])
        c = 0 if pad else min(c, left)
        left -= c
        counts.append(c)
    return lengths, counts


def _token_lengths(case):
    rng = random.Random(case["seed"])
    n = [_spread(rng, case["lo"], case["hi"]) for _ in range(case["rows"])]
    if case["lo"] < case["hi"] and case["rows"] > 1:
        n[rng.randrange(case["rows"])] = case["lo"]
    return n


def _prompt_lengths(case):
    """New tokens of each sequence, and all of them."""
    rng = random.Random(case["seed"])
    new = [_spread(rng, case["lo_new"], case["hi_new"]) for _ in range(case["n"])]
    if sum(new) == 0:
        new[0] = 1
    return new, [c + _spread(rng, case["lo_old"], case["hi_old"]) for c in new]


def _histories(case):
    """Tokens of each row's history, and how many of them are its prompt."""
    rng = random.Random(case["seed"])
    n = [_spread(rng, case["history"] // 3, case["history"]) for _ in range(case["n"])]
    return n, [rng.randint(0, x) for x in n]


# ---------------------------------------------------------------------------
# the inputs
# ---------------------------------------------------------------------------

def _normal(shape, g, dev, dtype, gain=1.0):
    return (torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16 if dtype == E4M3 else dtype) * gain).to(dtype)


def _i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _cache(case, lengths, g, dev):
    """A paged cache of sequences of ``lengths`` in pages of random order, with NaN behind each one's last token."""
    hkv, d, page, cache = case["hkv"], case["d"], case["page"], TYPES[case["cache"]]
    need = torch.tensor([-(-c // page) for c in lengths])
    total, width = int(need.sum()) + 3, max(1, int(need.max()))
    order = torch.randperm(total, generator=g, device=dev).int()
    first = (need.cumsum(0) - need).to(dev)
    col = torch.arange(width, device=dev)
    at = (first[:, None] + col).clamp_max(total - 1)
    s = dict(table=torch.where(col < need.to(dev)[:, None], order[at], torch.full_like(order[at], -1)), k_scale=None, v_scale=None)
    if cache == E4M3:
        s["k_scale"] = torch.rand(hkv, generator=g, device=dev) * 0.02 + 0.01
        s["v_scale"] = torch.rand(hkv, generator=g, device=dev) * 0.02 + 0.01
    n = _i32(lengths, dev)
    last = s["table"].gather(1, ((n.long() - 1).clamp_min(0) // page)[:, None])[:, 0]
    some = (n % page > 0).nonzero()[:, 0]
    tail = torch.arange(page, device=dev) >= (n % page)[some, None]
    to = last[some].long()[:, None].expand_as(tail)[tail], torch.arange(page, device=dev).expand_as(tail)[tail]
    for c in ("k_cache", "v_cache"):
        s[c] = _normal((total, hkv, page, d), g, dev, cache, 1.0 if cache != E4M3 else 48.0)
        s[c].view(torch.uint8 if cache == E4M3 else cache)[to[0], :, to[1]] = 0x7F if cache == E4M3 else float("nan")
    return s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return {"plan": _prepare_plan, "token": _prepare_token, "prompt": _prepare_prompt, "product": _prepare_product,
            "logits": _prepare_logits}[case["op"]](case, g, dev)


def _prepare_plan(case, g, dev):
    lengths, counts = _planned(case)
    page = case["page"]
    have = [-(-max(0, a) // page) for a in lengths]
    need = [-(-max(0, a + c) // page) for a, c in zip(lengths, counts)]
    taken, more = 5, sum(need) - sum(have)
    total = sum(have) + taken + more + 40
    order = torch.randperm(total, generator=g, device=dev).int()
    width = max(need) + 3
    table = torch.full((case["n"], width), -1, dtype=torch.int32)
    first = order[:sum(have)].cpu()
    at = 0
    for i, h in enumerate(have):
        table[i, :h] = first[at:at + h]
        at += h
    # the free pages, of which earlier steps have taken some; a short list cannot serve the step
    free = order[sum(have):]
    if case["short"] and more:
        free = free[:taken + more - 1].contiguous()
    return dict(case=case, lengths=_i32(lengths, dev), counts=None if case["step"] else _i32(counts, dev), table=table.to(dev), free=free,
                used=_i32([taken], dev))


def _prepare_token(case, g, dev):
    lengths = _token_lengths(case)
    s = _cache(case, lengths, g, dev)
    return dict(s, case=case, lengths=_i32(lengths, dev), q=_normal((case["rows"], case["hq"], case["d"]), g, dev, TYPES[case["x"]], 2.0))


def _prepare_prompt(case, g, dev):
    new, lengths = _prompt_lengths(case)
    s = _cache(case, lengths, g, dev)
    starts = [0]
    for c in new:
        starts.append(starts[-1] + c)
    # queries as the rows of a product that holds keys and values too
    qkv = _normal((starts[-1], case["hq"] + 2 * case["hkv"], case["d"]), g, dev, torch.bfloat16, 1.5)
    return dict(s, case=case, lengths=_i32(lengths, dev), starts=_i32(starts, dev), q=qkv[:, :case["hq"]])


def _prepare_product(case, g, dev):
    m, n, k = case["m"], case["n"], case["k"]
    x = _normal((m, k), g, dev, TYPES[case["x"]])
    x[:, :: 61] *= 12.0                                      # activations have channels that stand out
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    w = _normal((n, k), g, dev, E4M3, 90.0)
    w_scale = (torch.rand((nb, kb), generator=g, device=dev) + 0.5) * 2.0e-4
    return dict(case=case, x=x, w=w, w_scale=w_scale, residual=_normal((m, n), g, dev, TYPES[case["out"]]) if case["residual"] else None)


def _prepare_logits(case, g, dev):
    n, v = case["n"], case["vocab"]
    sizes, prompts = _histories(case)
    s = dict(case=case, logits=_normal((n, v), g, dev, TYPES[case["x"]], 3.0), tokens=None, lengths=None, prompts=None, repetition=None,
             presence=None, frequency=None, bias_ids=None, bias=None, mask=None)
    s["out"] = torch.empty_like(s["logits"])
    if case["penalties"]:
        width = max(1, case["history"])
        # texts repeat their frequent tokens
        u = torch.rand((n, width), generator=g, device=dev)
        s["tokens"] = ((v - 1) * u ** 3).int()
        s["lengths"], s["prompts"] = _i32(sizes, dev), _i32(prompts, dev)
        s["repetition"] = 1.0 + 0.3 * torch.rand(n, generator=g, device=dev)
        s["presence"] = 0.6 * torch.rand(n, generator=g, device=dev)
        s["frequency"] = 0.4 * torch.rand(n, generator=g, device=dev)
    if case["biases"]:
        # ids of a row are different ones; the last are unused
        b = min(case["biases"], v)
        ids = (torch.arange(b, device=dev) * (v // b) + torch.randint(0, v // b, (n, b), generator=g, device=dev)).int()
        ids[:, b - b // 8:] = -1
        s["bias_ids"], s["bias"] = ids, torch.randn((n, b), generator=g, device=dev) * 4.0
    if case["mask"]:
        words = torch.randint(-2 ** 31, 2 ** 31, (n, -(-v // 32)), generator=g, device=dev, dtype=torch.int64)
        words &= torch.randint(-2 ** 31, 2 ** 31, words.shape, generator=g, device=dev, dtype=torch.int64)
        s["mask"] = words.int()
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return {"plan": _plan, "token": _token, "prompt": _prompt, "product": _product, "logits": _logits}[s["case"]["op"]](s)


def _mk():
    import persistent_transformer_megakernel_gb300 as mk
    return mk


def _plan(s):
    case, lengths, table, free, used = s["case"], s["lengths"], s["table"], s["free"], s["used"]
    if own:
        return [*_mk().paged_plan(lengths, table, free, used, case["page"], counts=s["counts"], rows=case["rows"]), table]
    page, n, rows, dev = case["page"], case["n"], case["rows"], lengths.device
    live = lengths >= 0
    counts = live.int() if s["counts"] is None else torch.where(live, s["counts"].clamp_min(0), 0)
    have = (lengths.clamp_min(0).long() + page - 1) // page
    need = (lengths.clamp_min(0).long() + counts + page - 1) // page
    more = need - have
    first = used.long() + more.cumsum(0) - more
    left = free.shape[0] - used.long()
    fits = (more.sum() <= left) & (need.max() <= table.shape[1])
    if s["counts"] is not None:
        fits = fits & (counts.sum() <= rows)
    counts = torch.where(fits, counts, 0)
    col = torch.arange(table.shape[1], device=dev)
    new = fits & (col >= have[:, None]) & (col < need[:, None])
    at = (first[:, None] + col - have[:, None]).clamp(0, max(0, free.shape[0] - 1))
    table.copy_(torch.where(new, free[at], table))
    r = torch.arange(rows, device=dev)
    if s["counts"] is None:
        starts = torch.arange(n + 1, device=dev)
        seqs = torch.where(counts > 0, r, -1)
        slots = torch.where(counts > 0, lengths, -1)
    else:
        starts = torch.cat([torch.zeros(1, device=dev, dtype=torch.long), counts.cumsum(0)])
        seqs = torch.searchsorted(starts[1:].contiguous(), r, right=True).clamp_max(n - 1)
        there = r < starts[n]
        slots = torch.where(there, lengths[seqs] + r - starts[seqs], -1)
        seqs = torch.where(there, seqs, -1)
    totals = lengths + counts
    return [seqs.int(), slots.int(), starts.int(), totals.int(), torch.where(fits, used + more.sum(), used).int(), table]


def _token(s):
    q, case = s["q"], s["case"]
    if own:
        lse = torch.empty(q.shape[:2], device=q.device, dtype=torch.float32)
        out = _mk().paged_attention(q, s["k_cache"], s["v_cache"], s["table"], s["lengths"], window=case["window"], sinks=case["sinks"],
                                    k_scale=s["k_scale"], v_scale=s["v_scale"], lse=lse)
        return [out, lse]
    rows, hq, d = q.shape
    hkv, page = s["k_cache"].shape[1:3]
    n = s["lengths"].long()[:, None]
    # the first tokens, then the window behind them
    width = min(case["window"], max(1, case["hi"]))
    first = torch.arange(min(case["sinks"], max(1, case["hi"])), device=q.device)
    recent = (n - case["window"]).clamp_min(0) + torch.arange(width, device=q.device)
    pos = torch.cat([first.expand(rows, -1), recent], 1)
    there = pos < n
    there[:, :first.shape[0]] &= first < n - case["window"]
    at = s["table"].clamp_min(0).long().gather(1, (pos // page).clamp_max(s["table"].shape[1] - 1)), pos % page
    k = s["k_cache"][at[0], :, at[1]].float()                       # [rows][positions][hkv][d]
    v = s["v_cache"][at[0], :, at[1]].float()
    v.masked_fill_(~there[:, :, None, None], 0.0)
    if s["k_scale"] is not None:
        k *= s["k_scale"][:, None]
        v *= s["v_scale"][:, None]
    qs = q.float().view(rows, hkv, hq // hkv, d) * d ** -0.5
    z = torch.matmul(qs, k.permute(0, 2, 3, 1))
    z.masked_fill_(~there[:, None, None, :], -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, 1.0)
    lse = torch.log(total) + torch.where(torch.isinf(top), 0.0, top)
    return [out.view(rows, hq, d).to(q.dtype), lse.view(rows, hq)]


def _prompt(s):
    q, case = s["q"], s["case"]
    if own:
        lse = torch.empty(q.shape[:2], device=q.device, dtype=torch.float32)
        out = _mk().paged_prompt_attention(q, s["k_cache"], s["v_cache"], s["table"], s["starts"], s["lengths"], window=case["window"],
                                           sinks=case["sinks"], k_scale=s["k_scale"], v_scale=s["v_scale"], lse=lse)
        return [out, lse]
    rows, hq, d = q.shape
    hkv, page = s["k_cache"].shape[1:3]
    out, lse = torch.empty((rows, hq, d), device=q.device, dtype=q.dtype), torch.empty((rows, hq), device=q.device)
    new, lengths = _prompt_lengths(case)
    at = 0
    for i, (c, n) in enumerate(zip(new, lengths)):
        if c == 0:
            continue
        pages = s["table"][i, :-(-n // page)].long()
        k = s["k_cache"][pages].transpose(0, 1).reshape(hkv, -1, d)[:, :n].float()
        v = s["v_cache"][pages].transpose(0, 1).reshape(hkv, -1, d)[:, :n].float()
        if s["k_scale"] is not None:
            k *= s["k_scale"][:, None, None]
            v *= s["v_scale"][:, None, None]
        step = max(1, (1 << 29) // (hq * n))
        for a in range(0, c, step):
            b = min(c, a + step)
            qs = q[at + a:at + b].float().view(b - a, hkv, hq // hkv, d).permute(1, 2, 0, 3) * d ** -0.5
            z = torch.matmul(qs.reshape(hkv, -1, d), k.transpose(1, 2)).view(hkv, hq // hkv, b - a, n)
            own_pos = torch.arange(n - c + a, n - c + b, device=q.device)[:, None]
            p = torch.arange(n, device=q.device)
            seen = p <= own_pos
            if case["window"]:
                seen &= (p > own_pos - case["window"]) | (p < case["sinks"])
            z.masked_fill_(~seen, -math.inf)
            top = z.amax(-1, keepdim=True)
            e = torch.exp(z - top)
            total = e.sum(-1, keepdim=True)
            o = torch.matmul(e.view(hkv, -1, n), v).view(hkv, hq // hkv, b - a, d) / total
            out[at + a:at + b] = o.permute(2, 0, 1, 3).reshape(b - a, hq, d).to(q.dtype)
            lse[at + a:at + b] = (torch.log(total) + top)[..., 0].permute(2, 0, 1).reshape(b - a, hq)
        at += c
    return [out, lse]


def _product(s):
    x, w, w_scale, residual = s["x"], s["w"], s["w_scale"], s["residual"]
    dtype = TYPES[s["case"]["out"]]
    if own:
        mk = _mk()
        codes, scales = mk.quantize_fp8(x)
        return mk.matmul_fp8(codes, scales, w, w_scale, residual=residual, dtype=dtype)
    m, k = x.shape
    kb = w_scale.shape[1]
    blocks = torch.nn.functional.pad(x.float(), (0, kb * BLOCK - k)).view(m, kb, BLOCK)
    largest = blocks.abs().amax(-1)
    scales = torch.where(largest > 0, largest / torch.full_like(largest, 448.0), 1.0)
    xq = ((blocks / scales[..., None]).to(E4M3).float() * scales[..., None]).view(m, -1)[:, :k]
    wq = w.float() * w_scale.repeat_interleave(BLOCK, 0)[:w.shape[0]].repeat_interleave(BLOCK, 1)[:, :k]
    y = torch.matmul(xq, wq.t())
    if residual is not None:
        y = y + residual.float()
    return y.to(dtype)


def _logits(s):
    x = s["logits"]
    if own:
        return _mk().adjust_logits(x, **{f: s[f] for f in ("tokens", "lengths", "prompts", "repetition", "presence", "frequency", "bias_ids",
                                                           "bias", "mask", "out")})
    n, v = x.shape
    y = x.float()
    if s["tokens"] is not None:
        i = torch.arange(s["tokens"].shape[1], device=x.device)
        there = i < s["lengths"][:, None]
        ids = s["tokens"].long()
        seen = torch.zeros((n, v), device=x.device).scatter_add_(1, ids, there.float())
        made = torch.zeros((n, v), device=x.device).scatter_add_(1, ids, (there & (i >= s["prompts"][:, None])).float())
        r = s["repetition"][:, None]
        y = torch.where(seen > 0, torch.where(y > 0, y / r, y * r), y)
        y = y - s["frequency"][:, None] * made - torch.where(made > 0, s["presence"][:, None], 0.0)
    if s["bias_ids"] is not None:
        ok = s["bias_ids"] >= 0
        y = y.scatter_add(1, s["bias_ids"].clamp_min(0).long(), torch.where(ok, s["bias"], 0.0))
    if s["mask"] is not None:
        t = torch.arange(v, device=x.device)
        y = torch.where(s["mask"][:, t // 32] >> (t % 32) & 1 != 0, y, -math.inf)
    s["out"].copy_(y)
    return s["out"]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _seen(case, own_pos):
    """Tokens that the one at ``own_pos`` sees."""
    n = own_pos + 1
    return min(n, case["window"] + min(case["sinks"], max(0, n - case["window"]))) if case["window"] else n


def work(case):
    op = case["op"]
    if op == "plan":
        lengths, counts = _planned(case)
        page = case["page"]
        pages = sum(-(-max(0, a + c) // page) - -(-max(0, a) // page) for a, c in zip(lengths, counts))
        n = case["n"]
        return dict(bytes=4 * (n * (2 if case["step"] else 3) + n + 1 + 2 * case["rows"] + 2 * pages + 2), flops=8 * n + 4 * case["rows"])
    if op == "logits":
        n, v = case["n"], case["vocab"]
        b = 2 * n * v * SIZE[case["x"]] + (n * -(-v // 32) * 4 if case["mask"] else 0) + 8 * n * case["biases"]
        if case["penalties"]:
            b += 4 * sum(_histories(case)[0]) + 20 * n
        return dict(bytes=b, flops=4 * n * v)
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        b = m * k * SIZE[case["x"]] + n * k + 4 * -(-n // BLOCK) * -(-k // BLOCK) + m * n * SIZE[case["out"]] * (2 if case["residual"] else 1)
        return dict(bytes=b, flops=2 * m * n * k)
    hq, hkv, d, cs = case["hq"], case["hkv"], case["d"], SIZE[case["cache"]]
    if op == "token":
        seen = [_seen(case, n - 1) if n else 0 for n in _token_lengths(case)]
        rows, xs, read, pairs = case["rows"], SIZE[case["x"]], sum(seen), sum(seen)
    else:
        new, lengths = _prompt_lengths(case)
        rows, xs = sum(new), 2
        pairs = read = 0
        for c, n in zip(new, lengths):
            pairs += sum(_seen(case, p) for p in range(n - c, n))
            if c:
                read += min(n, c - 1 + _seen(case, n - c)) if case["window"] else n
    b = read * hkv * d * 2 * cs + rows * hq * (2 * d * xs + 4) + 4 * read // case["page"]
    return dict(bytes=b, flops=4 * pairs * hq * d)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "token": _exact_token, "prompt": _exact_prompt, "product": _exact_product,
            "logits": _exact_logits}[case["op"]](case, s)


def _exact_plan(case, s):
    lengths, counts = _planned(case)
    n, rows, page = case["n"], case["rows"], case["page"]
    table, free, used = s["table"].cpu().tolist(), s["free"].cpu().tolist(), int(s["used"])
    taken, changes = used, []
    for i in range(n):
        for t in range(max(0, lengths[i]), max(0, lengths[i]) + counts[i]):
            if t % page == 0:                                # the first token of a page
                changes.append((i, t // page, taken))
                taken += 1
    fits = taken <= len(free)
    if fits:
        for i, c, at in changes:
            table[i][c] = free[at]
    else:
        counts, taken = [0] * n, used
    seqs, slots, starts = [], [], [0]
    for i in range(n):
        if case["step"]:
            seqs.append(i if counts[i] else -1)
            slots.append(lengths[i] if counts[i] else -1)
            starts.append(i + 1)
        else:
            seqs += [i] * counts[i]
            slots += range(lengths[i], lengths[i] + counts[i])
            starts.append(len(seqs))
    seqs += [-1] * (rows - len(seqs))
    slots += [-1] * (rows - len(slots))
    dev = s["table"].device
    return [_i32(x, dev) for x in (seqs, slots, starts, [a + c for a, c in zip(lengths, counts)], [taken], table)]


def _held(s, i, n, page):
    """Keys and values of the first n tokens of sequence i: [hkv][n][d] in 64 bits."""
    out = []
    for c, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
        x = c[s["table"][i, : -(-n // page)].long()].permute(1, 0, 2, 3).flatten(1, 2)[:, :n].to(torch.float64)
        out.append(x if scale is None else x * scale.to(torch.float64)[:, None, None])
    return out


def _exact_token(case, s):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    out = torch.zeros((case["rows"], hq, d), device=s["q"].device, dtype=torch.float64)
    lse = torch.full((case["rows"], hq), -math.inf, device=s["q"].device, dtype=torch.float64)
    for b, n in enumerate(_token_lengths(case)):
        if n == 0:
            continue
        k, v = _held(s, b, n, case["page"])
        first, low = min(n, case["sinks"]), max(0, n - case["window"])
        if first < low:
            k, v = (torch.cat([x[:, :first], x[:, low:]], 1) for x in (k, v))
        z = torch.einsum("hgd,hnd->hgn", s["q"][b].to(torch.float64).view(hkv, -1, d), k) / math.sqrt(d)
        out[b] = torch.einsum("hgn,hnd->hgd", z.softmax(-1), v).reshape(hq, d)
        lse[b] = z.logsumexp(-1).reshape(hq)
    return [out, lse]


def _exact_prompt(case, s):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    q = s["q"]
    out = torch.zeros(q.shape, device=q.device, dtype=torch.float64)
    lse = torch.zeros(q.shape[:2], device=q.device, dtype=torch.float64)
    new, lengths = _prompt_lengths(case)
    row = 0
    for i, (c, n) in enumerate(zip(new, lengths)):
        if c == 0:
            continue
        k, v = _held(s, i, n, case["page"])
        for a in range(0, c, 512):
            b = min(c, a + 512)
            at = torch.arange(a, b, device=q.device) + n - c
            hi = n - c + b                                   # tokens behind the last of these rows are seen by none
            j = torch.arange(hi, device=q.device)
            hidden = j[None] > at[:, None]
            if case["window"]:
                hidden = hidden | ((at[:, None] - j[None] >= case["window"]) & (j[None] >= case["sinks"]))
            for h in range(hq):
                z = q[row + a:row + b, h].to(torch.float64) @ k[h // (hq // hkv), :hi].t() / math.sqrt(d)
                z[hidden] = -math.inf
                out[row + a:row + b, h] = z.softmax(-1) @ v[h // (hq // hkv), :hi]
                lse[row + a:row + b, h] = z.logsumexp(-1)
        row += c
    return [out, lse]


def _exact_product(case, s):
    """The scale of a block is the fp32 number next to largest / 448, a code the e4m3 number next to x / scale as an
    fp32 number (bf16 values over their scales are often half way between two codes)."""
    f = torch.float64
    m, n, k = case["m"], case["n"], case["k"]
    if 2 * m * n * k > 2e12:
        return None
    y = torch.zeros((m, n), device=s["x"].device, dtype=f) if s["residual"] is None else s["residual"].to(f)
    for b in range(-(-k // BLOCK)):
        x = s["x"][:, b * BLOCK:(b + 1) * BLOCK].to(f)
        scale = (x.abs().max(1, keepdim=True).values / 448).float().to(f)
        scale[scale == 0] = 1
        t = (x / scale).float().to(f)
        # half steps: three bits behind the leading one, and multiples of 2^-9 below 2^-6
        step = torch.exp2(torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -6))) - 3)
        t = (torch.round(t / step) * step).clamp(-448, 448) * scale
        w = s["w"][:, b * BLOCK:(b + 1) * BLOCK].to(f) * s["w_scale"][:, b].to(f).repeat_interleave(BLOCK)[:n, None]
        y += t @ w.t()
    return y


def _exact_logits(case, s):
    f = torch.float64
    n, v = case["n"], case["vocab"]
    y = s["logits"].to(f)
    sizes, prompts = _histories(case)
    for i in range(n):
        if s["tokens"] is not None and sizes[i]:
            past = s["tokens"][i, :sizes[i]].long()
            seen = past.unique()
            r = s["repetition"][i].to(f)
            a = y[i, seen]
            y[i, seen] = torch.where(a > 0, a / r, a * r)
            made, count = past[prompts[i]:].unique(return_counts=True)
            y[i, made] -= s["presence"][i].to(f) + s["frequency"][i].to(f) * count
        if s["bias_ids"] is not None:
            ok = s["bias_ids"][i] >= 0
            y[i, s["bias_ids"][i][ok].long()] += s["bias"][i][ok].to(f)
        if s["mask"] is not None:
            bits = (s["mask"][i].long()[:, None] >> torch.arange(32, device=y.device)) & 1
            y[i, bits.flatten()[:v] == 0] = -math.inf
    return y
