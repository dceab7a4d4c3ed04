"""Plain 64-bit forms of the operators of prompts and of a step's two ends, with their error bounds (see
serving_util for how a bound is counted)."""
import math

import torch

from serving_util import E4M3, F64, gather


def seen(n, first, last, window, sinks):
    """[last - first][n] truth values: whether the token at a position sees each of the first n tokens."""
    t, p = torch.arange(first, last)[:, None], torch.arange(n)[None]
    s = p <= t
    if window:
        s = s & ((p > t - window) | (p < sinks))
    return s


def masked_attention(q, k, v, see, scale, p_err, fp8):
    """``(out, lse, error, lse error)`` of rows q [rows][hq][d] over k, v [hkv][n][d] (64 bits) where ``see`` [rows][n]."""
    rows, hq, d = q.shape
    hkv, n = k.shape[:2]
    out, lse = torch.zeros((rows, hq, d), dtype=F64), torch.full((rows, hq), -math.inf, dtype=F64)
    err, lerr = torch.zeros((rows, hq, d), dtype=F64), torch.zeros((rows, hq), dtype=F64)
    some = see.any(1)
    for h in range(hq):
        kh, vh = k[h * hkv // hq], v[h * hkv // hq]
        # what a row does not see does not count, whatever it holds
        kh, vh = (torch.where(see.any(0)[:, None], x, 0.0) for x in (kh, vh))
        qh = q[:, h].to(F64)
        z = (qh @ kh.t()) * scale
        a = torch.where(see, (qh.abs() @ kh.abs().t()) * abs(scale), 0.0)
        z = torch.where(see, z, -math.inf)
        m = z.amax(1, keepdim=True)
        e = torch.exp(z - torch.where(torch.isinf(m), 0.0, m))
        l = e.sum(1, keepdim=True)
        w = torch.where(l == 0, 0.0, e / l)
        finite = torch.isfinite(vh)
        vf = torch.where(finite, vh, 0.0)
        o = w @ vf
        for p in (~finite).any(1).nonzero()[:, 0].tolist():  # an infinity or NaN is a result only where it is seen
            o = torch.where(see[:, p, None], o + torch.where(finite[p], 0.0, vh[p]), o)
        out[:, h] = torch.where(some[:, None], o, 0.0)
        lse[:, h] = torch.where(some, (m + l.log())[:, 0], -math.inf)
        # a score: d / 16 chained products of 16 terms; a weight: its rounding and 2^x to 2^-21; sums of n / 16 chained
        # products of 16 terms, each truncated, in tensor memory
        s_err = a.amax(1, keepdim=True) * 24 * 2.0 ** -23
        c = 2 * s_err + p_err + (64 + n / 8) * 2.0 ** -23
        # over an 8-bit cache weights are fp16 numbers, the largest 2^11 at least: small ones are rounded by half a step of
        # the subnormal numbers, 2^-25, which is 2^-36 of the largest
        err[:, h] = c * (w @ vf.abs()) + (n * 2.0 ** -36 * vf.abs().amax() if fp8 else 0.0)
        lerr[:, h] = (2 * s_err[:, 0] + (64 + n / 32) * 2.0 ** -23) + 2.0 ** -22 * torch.where(some, lse[:, h].abs(), 0.0)
    return out, lse, err, lerr


def prompt_attention(q, k_cache, v_cache, table, starts, lengths, scale, window=0, sinks=0, k_scale=None, v_scale=None):
    """The same of ``paged_prompt_attention``'s arguments (CPU tensors); rows of no sequence are NaN in ``out``."""
    rows, hq, d = q.shape
    fp8 = k_cache.dtype == E4M3
    out, lse = torch.full((rows, hq, d), math.nan, dtype=F64), torch.full((rows, hq), math.nan, dtype=F64)
    err, lerr = torch.zeros((rows, hq, d), dtype=F64), torch.zeros((rows, hq), dtype=F64)
    for i, n in enumerate(lengths.tolist()):
        a, b = int(starts[i]), int(starts[i + 1])
        if n < 0 or a == b:
            continue
        kv = []
        for c, s in ((k_cache, k_scale), (v_cache, v_scale)):
            x = gather(c, table[i], n) if n else torch.zeros((c.shape[1], 0, d), dtype=F64)
            kv.append(x if s is None else x * s.to(F64)[:, None, None])
        if n == 0:
            out[a:b], lse[a:b] = 0.0, -math.inf
            continue
        # a weight is rounded to bf16, or fp16 over an 8-bit cache: half a step
        r = masked_attention(q[a:b], *kv, seen(n, n - (b - a), n, window, sinks), scale, 2.0 ** -11 if fp8 else 2.0 ** -8, fp8)
        out[a:b], lse[a:b], err[a:b], lerr[a:b] = r
    return out, lse, err, lerr


def quantized(x):
    """``(codes, scales)`` of rows in 64 bits: a scale is the fp32 number next to largest / 448, a code the e4m3 number
    next to x / scale as an fp32 number."""
    m, k = x.shape
    kb = -(-k // 128)
    b = torch.nn.functional.pad(x.to(F64), (0, kb * 128 - k)).view(m, kb, 128)
    s = (torch.where(torch.isnan(b), 0.0, b.abs()).amax(-1) / 448).float().to(F64)
    s = torch.where(s > 0, s, 1.0)
    t = (b / s[..., None]).float().to(F64)
    step = torch.exp2(torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(t / step) * step).clamp(-448, 448).view(m, -1)[:, :k], s


def product(x, xs, w, ws):
    """``(y, error)`` of codes and scales (CPU)."""
    n, k = w.shape
    xd = x.to(F64) * xs.to(F64).repeat_interleave(128, 1)[:, :k]
    wd = w.to(F64) * ws.to(F64).repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    # a block: four products of 32 terms, each term truncated against the largest; the scales' product; a block's addition
    return xd @ wd.t(), (xd.abs() @ wd.abs().t()) * (4 * 33 + ws.shape[1] + 4) * 2.0 ** -23


def plan(lengths, counts, table, free, used, page, rows):
    """``(seqs, slots, starts, totals, used, table, fits)`` token by token (lists)."""
    n, step = len(lengths), counts is None
    take = [0 if a < 0 else 1 if step else max(0, counts[i]) for i, a in enumerate(lengths)]
    new, at, fits = [list(t) for t in table], used, step or sum(take) <= rows
    for i in range(n):
        for p in range(max(0, lengths[i]), max(0, lengths[i]) + take[i]):
            if p % page == 0:
                if at >= len(free) or p // page >= len(table[i]):
                    fits = False
                    break
                new[i][p // page] = free[at]
                at += 1
            elif p // page >= len(table[i]):
                fits = False
    if not fits:
        take, new, at = [0] * n, [list(t) for t in table], used
    seqs, slots, starts = [], [], [0]
    for i in range(n):
        here = list(range(lengths[i], lengths[i] + take[i]))
        if step:
            here = here or [-1]
        seqs += [i if p >= 0 else -1 for p in here]
        slots += here
        starts.append(len(seqs))
    if step:
        starts = list(range(n + 1))
    seqs += [-1] * (rows - len(seqs))
    slots += [-1] * (rows - len(slots))
    return seqs, slots, starts, [a + c for a, c in zip(lengths, take)], at, new, fits


def adjusted(x, tokens=None, lengths=None, prompts=None, repetition=None, presence=None, frequency=None, bias_ids=None, bias=None, mask=None):
    """``(y, error)`` of ``adjust_logits`` (CPU tensors), rows of negative length NaN."""
    n, v = x.shape
    y, size = x.to(F64), x.to(F64).abs()
    for i in range(n):
        count = (tokens.shape[1] if tokens is not None else 0) if lengths is None else int(lengths[i])
        if count < 0:
            y[i] = math.nan
            continue
        past = [] if tokens is None else tokens[i, :count].tolist()
        first = 0 if prompts is None else int(prompts[i])
        for t in sorted(set(past)):
            if not 0 <= t < v:
                continue
            if repetition is not None:
                r = float(repetition[i])
                y[i, t] = y[i, t] / r if y[i, t] > 0 else y[i, t] * r
                size[i, t] = torch.maximum(size[i, t], y[i, t].abs())
            c = past[first:].count(t)
            if c:
                f, p = (0.0 if a is None else float(a[i]) for a in (frequency, presence))
                y[i, t] -= f * c + p
                size[i, t] += abs(f * c) + abs(p)
        if bias_ids is not None:
            for t, b in zip(bias_ids[i].tolist(), bias[i].tolist()):
                if 0 <= t < v:
                    y[i, t] += b
                    size[i, t] += abs(b)
        if mask is not None:
            bits = (mask[i].long()[:, None] >> torch.arange(32)) & 1
            y[i, bits.flatten()[:v] == 0] = -math.inf
    # a quotient, a product, and an addition for each penalty and bias
    return y, torch.where(torch.isfinite(size), size, 0.0) * (6 + (0 if bias_ids is None else bias_ids.shape[1])) * 2.0 ** -24
