"""``paged_prompt_attention`` against its definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

import prompt_util as P
import serving_util as U

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _cache(lengths, hkv, d, page, cache, seed, spread=1.0):
    rng, g = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
    table, total = U.pages([max(0, n) for n in lengths], page, rng)
    kc, vc = (torch.randn((total, hkv, page, d), generator=g) * spread for _ in range(2))
    scales = None, None
    if cache == E4M3:
        kc, vc = kc * 40, vc * 40
        scales = torch.rand(hkv, generator=g) * 0.02 + 0.01, torch.rand(hkv, generator=g) * 0.02 + 0.01
    return kc.to(cache), vc.to(cache), table, *scales


def _run(q, kc, vc, table, starts, lengths, window=0, sinks=0, ks=None, vs=None, scale=None, out=None, stream=None):
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    s = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = mk.paged_prompt_attention(q.cuda(), c(kc), c(vc), c(table), c(starts), c(lengths), window=window, sinks=sinks, k_scale=c(ks), v_scale=c(vs),
                                    scale=scale, out=torch.full_like(q.cuda(), 7.0) if out is None else out, lse=lse, status=s, stream=stream)
    return out, lse, int(s)


def _check(new, lengths, hq, hkv, d, page, cache=BF16, window=0, sinks=0, seed=0, spread=1.0):
    kc, vc, table, ks, vs = _cache(lengths, hkv, d, page, cache, seed, spread)
    # nothing that is not a token of a sequence is a number
    for c in (kc, vc):
        raw = c.view(torch.uint8) if cache == E4M3 else c
        used = torch.zeros(raw.shape[0], page, dtype=torch.bool)
        for i, n in enumerate(lengths):
            for t in range(max(0, n)):
                used[table[i, t // page], t % page] = True
        raw.permute(0, 2, 1, 3)[~used] = 0x7F if cache == E4M3 else math.nan
    starts = torch.tensor([0] + np.cumsum(new).tolist(), dtype=torch.int32)
    rows = int(starts[-1]) + 3
    q = (torch.randn((rows, hq, d), generator=torch.Generator().manual_seed(seed + 1)) * 1.5).to(BF16)
    ln = torch.tensor(lengths, dtype=torch.int32)
    out, lse, status = _run(q, kc, vc, table, starts, ln, window, sinks, ks, vs)
    want, wl, err, el = P.prompt_attention(q, kc, vc, table, starts, ln, d ** -0.5, window, sinks, ks, vs)
    assert status == 0
    there = torch.zeros(rows, dtype=torch.bool)
    for i, n in enumerate(lengths):
        there[starts[i]:starts[i + 1]] = n >= 0
    assert (out.cpu()[~there] == 7).all() and (lse.cpu()[~there] == 7).all()
    U.assert_within(out.cpu()[there], want[there], (U.half_step(BF16, want) + err)[there], "out")
    U.assert_within(lse.cpu()[there], wl[there], el[there], "lse")


# every head group from one to more than a tile holds, both widths and caches
@pytest.mark.parametrize("hq,hkv,d,cache", [(1, 1, 64, BF16), (2, 2, 128, BF16), (16, 8, 128, BF16), (6, 2, 128, E4M3), (8, 2, 64, E4M3), (5, 1, 64, BF16),
                                            (16, 1, 128, E4M3), (130, 1, 64, BF16), (7, 7, 64, E4M3)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
def test_heads(hq, hkv, d, cache, window, sinks):
    _check([70, 1, 200], [70, 90, 333], hq, hkv, d, 16, cache, window, sinks)


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("page", [1, 7, 16, 24, 128, 200])
def test_pages(page, cache):
    _check([33, 130, 5], [33, 131, 400], 4, 2, 64 if page % 2 else 128, page, cache, window=0 if page < 24 else 129, sinks=5)


@pytest.mark.parametrize("new,lengths", [([1], [1]), ([127], [127]), ([128], [128]), ([129], [129]), ([256], [300]), ([257], [257]), ([1], [2500]),
                                         ([5, 0, 3], [3000, 10, 3]), ([0, 0], [0, 4]), ([3], [0]), ([4, 9], [2, 9]), ([640], [4000]),
                                         ([10, 20, 30], [10, -1, 30])])
def test_lengths(new, lengths):
    _check(new, lengths, 4, 2, 128, 16)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (128, 0), (127, 128), (300, 4), (1000, 130), (5000, 9), (64, 5000)])
@pytest.mark.parametrize("d,cache", [(64, BF16), (128, E4M3)])
def test_windows(window, sinks, d, cache):
    _check([700, 40], [1500, 2100], 4, 2, d, 24, cache, window, sinks, seed=3)


def test_many_sequences():
    rng = np.random.default_rng(4)
    new = rng.integers(0, 40, 150).tolist()
    _check(new, [c + int(x) for c, x in zip(new, rng.integers(0, 300, 150))], 4, 2, 64, 16, window=100, sinks=2)


def test_wide_scores():
    # maxima that keep growing along a row: sums and results are rescaled again and again
    _check([300], [1200], 2, 1, 64, 16, spread=30.0)
    _check([300], [1200], 2, 1, 128, 16, E4M3, spread=3.0)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-30, 3.0])
@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_scales(scale, cache):
    kc, vc, table, ks, vs = _cache([150], 2, 64, 16, cache, 0, 0.3)
    q, starts, n = (torch.randn((150, 4, 64)) * 0.5).to(BF16), torch.tensor([0, 150], dtype=torch.int32), torch.tensor([150], dtype=torch.int32)
    out, lse, _ = _run(q, kc, vc, table, starts, n, ks=ks, vs=vs, scale=scale)
    want, wl, err, el = P.prompt_attention(q, kc, vc, table, starts, n, float(torch.tensor(scale)), 0, 0, ks, vs)
    U.assert_within(out, want, U.half_step(BF16, want) + err, "out")
    U.assert_within(lse, wl, el, "lse")


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("long", [False, True])
def test_what_a_row_does_not_see_may_be_anything(cache, long):
    # tokens with NaN and infinities between others: rows before them, and rows whose window has passed them, are finite
    n, count, window = (2600, 2600, 400) if long else (200, 200, 60)
    kc, vc, table, ks, vs = _cache([n], 2, 64, 16, cache, 1)
    kr, vr = (c.view(torch.uint8) if cache == E4M3 else c for c in (kc, vc))
    bad = 0x7F if cache == E4M3 else math.nan
    for p, where in ((n // 2, vr), (n // 2 + 3, kr), (n - 2, vr)):
        where[table[0, p // 16], :, p % 16] = bad
    if cache == BF16:
        vc[table[0, (n // 4) // 16], 0, (n // 4) % 16, 5] = math.inf
    q = torch.randn((count, 4, 64)).to(BF16)
    starts, ln = torch.tensor([0, count], dtype=torch.int32), torch.tensor([n], dtype=torch.int32)
    out, lse, _ = _run(q, kc, vc, table, starts, ln, window, 4, ks, vs)
    k, v = (U.gather(c, table[0], n) * (1.0 if s is None else s.double()[:, None, None]) for c, s in ((kc, ks), (vc, vs)))
    see = P.seen(n, 0, n, window, 4)
    nan_k = torch.isnan(k).any(2).any(0)
    hit = (see & nan_k[None]).any(1)
    want, wl, err, el = P.masked_attention(q[~hit], torch.where(nan_k[:, None], 0.0, k), v, (see & ~nan_k)[~hit], 64 ** -0.5,
                                           2.0 ** -11 if cache == E4M3 else 2.0 ** -8, cache == E4M3)
    assert hit.any() and torch.isfinite(want).any()
    U.assert_within(out.cpu()[~hit], want, U.half_step(BF16, want) + err, "out")
    U.assert_within(lse.cpu()[~hit], wl, el, "lse")
    assert torch.isnan(out.cpu()[hit]).all()


def test_values_near_the_largest():
    n = 1200
    kc, vc, table, _, _ = _cache([n], 1, 64, 16, BF16, 2)
    big = torch.finfo(BF16).max
    vc = torch.where(torch.rand(vc.shape) < 0.5, vc, torch.full_like(vc, big))
    vc[:, :, :, :7] = big
    q = (torch.randn((n, 2, 64)) * 0.3).to(BF16)
    starts, ln = torch.tensor([0, n], dtype=torch.int32), torch.tensor([n], dtype=torch.int32)
    out, lse, _ = _run(q, kc, vc, table, starts, ln)
    want, wl, err, el = P.prompt_attention(q, kc, vc, table, starts, ln, 64 ** -0.5)
    # a result next to the type's largest may round to either side of it
    near = want.abs() + err + U.half_step(BF16, want) >= big
    assert near.any() and not near.all()
    got = out.cpu().double()
    assert (got[near] >= big * (1 - 2.0 ** -7)).all()
    U.assert_within(torch.where(near, 0.0, got), torch.where(near, 0.0, want), U.half_step(BF16, want) + err, "out")


def test_queries_without_numbers():
    kc, vc, table, _, _ = _cache([100], 2, 64, 16, BF16, 3)
    q = torch.randn((100, 4, 64)).to(BF16)
    want = _run(q, kc, vc, table, torch.tensor([0, 100], dtype=torch.int32), torch.tensor([100], dtype=torch.int32))[0]
    q[17, 2, 3], q[40, 0, 0] = math.nan, math.inf
    got = _run(q, kc, vc, table, torch.tensor([0, 100], dtype=torch.int32), torch.tensor([100], dtype=torch.int32))[0]
    assert torch.isnan(got[17, 2]).all() and torch.isnan(got[40, 0]).all()
    want[17, 2], want[40, 0] = 0, 0
    got[17, 2], got[40, 0] = 0, 0
    assert torch.equal(got, want)


@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_bad_pages_lengths_and_starts(cache):
    new, lengths = [40, 30, 20, 10], [40, 1300, 20, 10]
    kc, vc, table, ks, vs = _cache(lengths, 2, 64, 16, cache, 5)
    starts = torch.tensor([0, 40, 70, 90, 100], dtype=torch.int32)
    q = torch.randn((100, 4, 64)).to(BF16)
    ln = torch.tensor(lengths, dtype=torch.int32)
    good = _run(q, kc, vc, table, starts, ln, ks=ks, vs=vs)
    assert good[2] == 0
    bad = table.clone()
    bad[0, 1] = -1                                          # tokens 16 .. 31 of the first
    bad[1, 60] = kc.shape[0]
    out, lse, status = _run(q, kc, vc, bad, starts, ln, ks=ks, vs=vs)
    assert status == -10
    assert torch.isnan(out[16:70]).all() and torch.isnan(lse[16:70]).all()
    for i in (slice(0, 16), slice(70, 100)):
        assert torch.equal(out[i], good[0][i]) and torch.equal(lse[i], good[1][i])
    # a sequence longer than its row of the table
    far = ln.clone()
    far[2] = 2 ** 31 - 1
    out, lse, status = _run(q, kc, vc, table, starts, far, ks=ks, vs=vs)
    assert status == -10 and torch.isnan(out[70:90]).all() and torch.equal(out[:70], good[0][:70]) and torch.equal(out[90:], good[0][90:])
    # starts that decrease or leave the rows: those sequences are skipped
    odd = torch.tensor([0, 40, 30, 101, 100], dtype=torch.int32)
    out, lse, status = _run(q, kc, vc, table, odd, ln, ks=ks, vs=vs)
    assert status == -10 and torch.equal(out[:40], good[0][:40]) and (out[40:] == 7).all()


def test_layouts_in_place_and_on_another_stream():
    # heads inside slots, keys and values of a page together; queries as part of a product's rows; out is q
    lengths, new, hkv, d, page = [90, 300], [90, 100], 2, 64, 16
    table, total = U.pages(lengths, page, np.random.default_rng(0))
    g = torch.Generator().manual_seed(0)
    both = torch.randn((total, 2, page, hkv, d), generator=g).to(BF16)
    kc, vc = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    starts, ln = torch.tensor([0, 90, 190], dtype=torch.int32), torch.tensor(lengths, dtype=torch.int32)
    qkv = torch.randn((190, 8, d), generator=g).to(BF16)
    want, wl, err, el = P.prompt_attention(qkv[:, 1:5], kc, vc, table, starts, ln, d ** -0.5)
    dev = both.cuda()
    rows = qkv.cuda()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = mk.paged_prompt_attention(rows[:, 1:5], dev[:, 0].transpose(1, 2), dev[:, 1].transpose(1, 2), table.cuda(), starts.cuda(), ln.cuda(),
                                    out=rows[:, 1:5], stream=stream)
    stream.synchronize()
    U.assert_within(got, want, U.half_step(BF16, want) + err, "out")
    assert torch.equal(rows[:, 0].cpu(), qkv[:, 0]) and torch.equal(rows[:, 5:].cpu(), qkv[:, 5:])


def test_captured_and_repeated():
    # one capture serves other lengths; two graphs and a plain call give the same bits
    hkv, d, page = 2, 128, 16
    kc, vc, table, _, _ = _cache([5000, 700], hkv, d, page, BF16, 6)
    kc, vc, table = kc.cuda(), vc.cuda(), table.cuda()
    q = torch.randn((400, 4, d)).to(BF16).cuda()
    starts, ln = torch.tensor([0, 0, 0], dtype=torch.int32, device="cuda"), torch.tensor([1, 1], dtype=torch.int32, device="cuda")
    out = [torch.zeros_like(q) for _ in range(2)]
    torch.cuda.synchronize()
    graphs = []
    for o in out:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mk.paged_prompt_attention(q, kc, vc, table, starts, ln, out=o)
        graphs.append(g)
    for a, b, n0, n1 in ((5, 400, 5000, 700), (400, 400, 4999, 3), (0, 390, 0, 500)):
        starts.copy_(torch.tensor([0, a, b])), ln.copy_(torch.tensor([n0, n1]))
        for g in graphs:
            g.replay()
        plain = torch.zeros_like(q)
        mk.paged_prompt_attention(q, kc, vc, table, starts, ln, out=plain)
        assert torch.equal(out[0][:b], plain[:b]) and torch.equal(out[1][:b], plain[:b])
        want, _, err, _ = P.prompt_attention(q[:b].cpu(), kc.cpu(), vc.cpu(), table.cpu(), starts.cpu(), ln.cpu(), d ** -0.5)
        U.assert_within(plain[:b], want, U.half_step(BF16, want) + err, "out")


def test_nothing_to_do():
    kc, vc, table, _, _ = _cache([20], 2, 64, 16, BF16, 7)
    kc, vc, table = kc.cuda(), vc.cuda(), table.cuda()
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    assert mk.paged_prompt_attention(torch.zeros((0, 4, 64), dtype=BF16, device="cuda"), kc, vc, table, z(2), z(1)).shape == (0, 4, 64)
    q = torch.ones((3, 4, 64), dtype=BF16, device="cuda")
    assert mk.paged_prompt_attention(q, kc, vc, table[:0], z(1), z(0), out=q) is q and (q == 1).all()


def test_rows_behind_an_offset_of_32_bits():
    # a cache of more than 2^32 bytes and rows of q more than 2^31 elements apart
    page, hkv, d = 16, 8, 128
    total = (1 << 32) // (page * hkv * d * 2) + 40
    kc = torch.zeros((total, hkv, page, d), dtype=BF16, device="cuda")
    vc = torch.zeros_like(kc)
    order = torch.tensor([[total - 1, 3, total - 5, total - 2]], dtype=torch.int32)
    some = torch.randn((2, 4, hkv, page, d)).to(BF16)
    kc[order[0].long()], vc[order[0].long()] = some[0].cuda(), some[1].cuda()
    q = torch.randn((50, 16, d)).to(BF16)
    starts, ln = torch.tensor([0, 50], dtype=torch.int32), torch.tensor([60], dtype=torch.int32)
    wide = torch.zeros(49 * (1 << 26) + 16 * d, dtype=BF16, device="cuda")
    view = wide.as_strided((50, 16, d), (1 << 26, d, 1))
    view.copy_(q)
    got = mk.paged_prompt_attention(view, kc, vc, order.cuda(), starts.cuda(), ln.cuda(), out=view)
    want, _, err, _ = P.prompt_attention(q, some[0], some[1], torch.arange(4, dtype=torch.int32)[None], starts, ln, d ** -0.5)
    U.assert_within(got, want, U.half_step(BF16, want) + err, "out")
