"""``paged_attention`` with first tokens that a window leaves visible, and next to ``paged_prompt_attention``."""
import math

import numpy as np
import pytest
import torch

import prompt_util as P
import serving_util as U

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _expected(q, kc, vc, table, lengths, window, sinks, ks, vs):
    """The definition row by row, over the tokens that are seen; errors as of plain attention over so many."""
    n, hq, d = q.shape
    outs = []
    for b in range(n):
        length = int(lengths[b])
        see = P.seen(length, length - 1, length, window, sinks)[0] if length > 0 else torch.zeros(0, dtype=torch.bool)
        rows = see.nonzero()[:, 0]
        k, v = (U.gather(c, table[b], length)[:, rows] if length > 0 else torch.zeros((kc.shape[1], 0, d), dtype=U.F64) for c in (kc, vc))
        # as a cache of 64-bit values of one page
        page = max(1, len(rows))
        fit = lambda x: torch.cat([x, torch.zeros((x.shape[0], page - x.shape[1], d), dtype=U.F64)], 1)[None]  # noqa: E731
        one = fit(k), fit(v)
        if kc.dtype == E4M3:
            one = tuple(x.to(E4M3) for x in one)
        outs.append(U.attention(q[b:b + 1], *one, torch.zeros((1, 1), dtype=torch.int32), torch.tensor([len(rows)]), d ** -0.5, 0, ks, vs))
    return [torch.cat(x) for x in zip(*outs)]


@pytest.mark.parametrize("x,cache", [(F32, BF16), (BF16, BF16), (F32, E4M3), (BF16, E4M3)])
@pytest.mark.parametrize("hq,hkv,d,page", [(4, 2, 64, 16), (16, 1, 128, 24), (3, 3, 128, 1)])
@pytest.mark.parametrize("lengths,window,sinks", [([700], 100, 4), ([700], 100, 130), ([33, 0, 1, 200, 2000, 901], 64, 1), ([33, 0, 1, 200, 2000, 901], 700, 40),
                                                  ([5000, 3000], 1100, 17), ([100, 101, 102], 100, 1), ([300], 1, 1), ([120, 500], 50, 4000)])
def test_first_tokens_stay_visible(x, cache, hq, hkv, d, page, lengths, window, sinks):
    rng, g = np.random.default_rng(1), torch.Generator().manual_seed(1)
    table, total = U.pages(lengths, page, rng)
    kc, vc = (torch.randn((total, hkv, page, d), generator=g) for _ in range(2))
    ks = vs = None
    if cache == E4M3:
        kc, vc, ks, vs = kc * 40, vc * 40, torch.rand(hkv, generator=g) * 0.02 + 0.01, torch.rand(hkv, generator=g) * 0.02 + 0.01
    kc, vc = kc.to(cache), vc.to(cache)
    ln = torch.tensor(lengths, dtype=torch.int32)
    # tokens between the first ones and the window are no numbers
    hidden = (kc.clone(), vc.clone())
    for c in hidden:
        raw = c.view(torch.uint8) if cache == E4M3 else c
        for b, n in enumerate(lengths):
            for t in range(sinks, max(sinks, n - window)):
                raw[table[b, t // page], :, t % page] = 0x7F if cache == E4M3 else math.nan
    q = (torch.randn((len(lengths), hq, d), generator=g) * 1.5).to(x)
    want, wl, err, el = _expected(q, kc, vc, table, ln, window, sinks, ks, vs)
    lse, s = torch.zeros(q.shape[:2], device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    got = mk.paged_attention(c(q), c(hidden[0]), c(hidden[1]), c(table), c(ln), window=window, sinks=sinks, k_scale=c(ks), v_scale=c(vs), lse=lse, status=s)
    assert int(s) == 0
    U.assert_within(got, want, U.half_step(x, want) + err, "out")
    U.assert_within(lse, wl, el, "lse")


def test_without_a_window_nothing_changes():
    g = torch.Generator().manual_seed(2)
    table, total = U.pages([900, 40], 16, np.random.default_rng(2))
    kc, vc = (torch.randn((total, 2, 16, 128), generator=g).to(BF16).cuda() for _ in range(2))
    q, ln = torch.randn((2, 4, 128), generator=g).to(BF16).cuda(), torch.tensor([900, 40], dtype=torch.int32, device="cuda")
    a = mk.paged_attention(q, kc, vc, table.cuda(), ln)
    assert torch.equal(a, mk.paged_attention(q, kc, vc, table.cuda(), ln, sinks=7))
    b = mk.paged_attention(q, kc, vc, table.cuda(), ln, window=300)
    assert torch.equal(b, mk.paged_attention(q, kc, vc, table.cuda(), ln, window=300, sinks=0)) and not torch.equal(a, b)
    assert torch.equal(b[1], mk.paged_attention(q, kc, vc, table.cuda(), ln, window=300, sinks=9)[1])


def test_a_bad_page_among_the_first_tokens_only_counts_where_it_is_seen():
    table, total = U.pages([600, 600], 16, np.random.default_rng(3))
    kc, vc = (torch.randn((total, 2, 16, 64)).to(BF16).cuda() for _ in range(2))
    q, ln = torch.randn((2, 2, 64)).to(BF16).cuda(), torch.tensor([600, 600], dtype=torch.int32, device="cuda")
    table[0, 0], table[1, 5] = -1, -1
    s = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mk.paged_attention(q, kc, vc, table.cuda(), ln, window=100, sinks=4, status=s)
    assert int(s) == -10 and torch.isnan(got[0]).all() and torch.isfinite(got[1]).all()


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 4)])
def test_a_prompt_and_its_tokens_one_by_one(cache, window, sinks):
    # both forms compute the same rows: within the sum of their bounds of each other
    n, hq, hkv, d = 700, 4, 2, 128
    g = torch.Generator().manual_seed(4)
    table, total = U.pages([n], 16, np.random.default_rng(4))
    kc, vc = ((torch.randn((total, hkv, 16, d), generator=g) * (40 if cache == E4M3 else 1)).to(cache).cuda() for _ in range(2))
    ks = vs = torch.full((hkv,), 0.025, device="cuda") if cache == E4M3 else None
    q = torch.randn((n, hq, d), generator=g).to(BF16).cuda()
    whole = mk.paged_prompt_attention(q, kc, vc, table.cuda(), torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                                      torch.tensor([n], dtype=torch.int32, device="cuda"), window=window, sinks=sinks, k_scale=ks, v_scale=vs)
    rows = mk.paged_attention(q, kc, vc, table.cuda().expand(n, -1), torch.arange(1, n + 1, dtype=torch.int32, device="cuda"), window=window, sinks=sinks,
                              k_scale=ks, v_scale=vs)
    s = None if ks is None else ks.cpu()
    want, _, err, _ = P.prompt_attention(q.cpu(), kc.cpu(), vc.cpu(), table, torch.tensor([0, n]), torch.tensor([n]), d ** -0.5, window, sinks, s, s)
    U.assert_within(whole, rows.cpu().double(), 2 * (U.half_step(BF16, want) + err) * 1.01, "both forms")
