"""Plain 64-bit forms of the paged-cache and 4-bit operators and their error
bounds, shared by the tests.

Bounds.  A result rounded once to type T is off by at most half a step,
``finfo(T).eps / 2`` of its value (e4m3: at least half of its smallest step,
2^-10).  What comes before it is fp32: every sum of n products whose partial
sums stay below A is off by at most n 2^-23 A (2^-23, not 2^-24: matrix products
truncate).  The functions return that part per element, as a multiple of the
sum of absolute products the element is made of.
"""
import math

import torch

F64 = torch.float64
E4M3 = torch.float8_e4m3fn


def half_step(dtype, want):
    e = torch.finfo(dtype).eps / 2
    t = want.abs() * e
    return t.clamp_min(2.0 ** -10) if dtype == E4M3 else t


def assert_within(got, want, tol, what):
    got, want = got.detach().to(F64).cpu(), want.cpu()
    tol = tol.cpu() if isinstance(tol, torch.Tensor) else torch.full_like(want, tol)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fine), what + ": finite in other places"
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what + ": NaN in other places"
    inf = ~fine & ~torch.isnan(want)
    assert torch.equal(got[inf], want[inf]), what + ": another infinity"
    over = ((got - want).abs() - tol)[fine]
    assert over.numel() == 0 or float(over.max()) <= 0, "%s: %.3g over its bound of %.3g" % (
        what, float(over.max()), float(tol.expand_as(want)[fine][over.argmax()]))


def gather(cache, table, n):
    """The first n slots of the sequence whose pages ``table`` names: [kv heads][n][d] in 64 bits."""
    page = cache.shape[2]
    pages = table[:-(-n // page)].long()
    x = cache.view(torch.uint8 if cache.dtype == E4M3 else cache.dtype)[pages].view(cache.dtype)
    return x.transpose(0, 1).reshape(cache.shape[1], -1, cache.shape[3])[:, :n].to(F64)


def attention(q, k_cache, v_cache, table, lengths, scale, window=0, k_scale=None, v_scale=None):
    """``(out, lse, error, lse error)`` of rows with length >= 0 (zeros elsewhere): CPU tensors in, 64 bits out."""
    n, hq, d = q.shape
    hkv = k_cache.shape[1]
    fp8 = k_cache.dtype == E4M3
    out, lse = torch.zeros((n, hq, d), dtype=F64), torch.full((n, hq), -math.inf, dtype=F64)
    err, lerr = torch.zeros((n, hq, d), dtype=F64), torch.zeros((n, hq), dtype=F64)
    for b in range(n):
        length = int(lengths[b])
        lo = max(0, length - window) if window else 0
        if length <= lo:
            continue
        k = gather(k_cache, table[b], length)[:, lo:]
        v = gather(v_cache, table[b], length)[:, lo:]
        if k_scale is not None:
            k, v = k * k_scale.to(F64)[:, None, None], v * v_scale.to(F64)[:, None, None]
        qb = q[b].to(F64).view(hkv, hq // hkv, d)
        z = torch.einsum("hgd,hnd->hgn", qb, k) * scale
        a = torch.einsum("hgd,hnd->hgn", qb.abs(), k.abs()) * abs(scale)
        m = z.amax(-1, keepdim=True)
        e = torch.exp(z - m)
        l = e.sum(-1, keepdim=True)
        out[b] = torch.einsum("hgn,hnd->hgd", e / l, v).reshape(hq, d)
        lse[b] = (m + l.log())[..., 0].reshape(hq)
        # a score: up to 8 chained products of 16 terms and 8 roundings; e4m3 caches round an fp32 query to 22 bits
        s_err = a.amax(-1, keepdim=True) * (24 * 2.0 ** -23 + (2.0 ** -22 if fp8 else 0))
        tiles = (length - lo) / 16 + 2
        # a probability's terms.  bf16 cache and query: 8 bits truncated leave less than 2^-7, of which 8 rounded bits
        # miss 2^-8 at most: 2^-15; three terms hold all 24 bits.  e4m3 cache: fp16 terms of 11 bits, one with a bf16 query
        p_err = (2.0 ** -11 if q.dtype == torch.bfloat16 else 2.0 ** -22) if fp8 else 2.0 ** -15 if q.dtype == torch.bfloat16 else 2.0 ** -23
        # 2^x to 2^-21, a tile's sum of 96 products at most, a multiply-add a tile, three joins
        c = 2 * s_err + p_err + (16 + 96 + tiles) * 2.0 ** -23
        err[b] = (c * torch.einsum("hgn,hnd->hgd", e / l, v.abs())).reshape(hq, d)
        lerr[b] = (2 * s_err[..., 0] + (64 + tiles) * 2.0 ** -23).reshape(hq) + 2.0 ** -22 * lse[b].abs()
    return out, lse, err, lerr


def rotary(pos, d, theta=1e6):
    i = torch.arange(d // 2, dtype=F64)
    return pos.to(F64)[..., None] * theta ** (-2 * i / d)


def pair_streams(d, sections, interleaved):
    out = []
    for i in range(d // 2):
        if interleaved:
            out.append(i % 3 if i % 3 and i < 3 * sections[i % 3] else 0)
        else:
            out.append(0 if i < sections[0] else 1 if i < sections[0] + sections[1] else 2)
    return out


def turned(x, gain, angle, eps):
    """``(value, error)`` of heads [n][heads][d] normalised by ``gain`` and turned by ``angle`` [n][d / 2] (each or both None)."""
    x = x.to(F64)
    d = x.shape[-1]
    err = x.abs() * 2.0 ** -24
    if gain is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gain.to(F64)
        err = x.abs() * (d + 16) * 2.0 ** -24       # a sum of d squares, a root, a quotient, two products
    if angle is not None:
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        a, b = x[..., :d // 2], x[..., d // 2:]
        ea, eb = err[..., :d // 2], err[..., d // 2:]
        both = (a.abs() + b.abs()) * 2.0 ** -22 + ea + eb        # fp32 cos and sin, two products, a sum
        return torch.cat([a * c - b * s, b * c + a * s], -1), torch.cat([both, both], -1)
    return x, err


def dequantize(codes, scales, zeros=None):
    """The weights of ``quantize_q4`` in 64 bits."""
    n, k = codes.shape[0], codes.shape[1] * 2
    c = torch.empty((n, k), dtype=F64)
    c[:, 0::2], c[:, 1::2] = (codes.cpu() & 15).to(F64), (codes.cpu() >> 4).to(F64)
    group = k // scales.shape[1]
    z = 8.0 if zeros is None else zeros.cpu().to(F64).repeat_interleave(group, 1)
    return (c - z) * scales.cpu().to(F64).repeat_interleave(group, 1)


def pages(lengths, page, rng, spare=2):
    """A random page table (a CPU int32 tensor) for sequences of ``lengths``, unused entries -1, and the page count."""
    need = [max(0, -(-int(n) // page)) for n in lengths]
    total = sum(need) + spare
    order = rng.permutation(total)
    table = torch.full((len(need), max(need + [1])), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.from_numpy(order[at:at + n].astype("int32"))
        at += n
    return table, total
