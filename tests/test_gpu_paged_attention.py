"""``paged_attention`` against its definition in 64 bits: head layouts, types,
page sizes, lengths from none to thousands, windows, strides, what lies behind a
row's last token, and how the call behaves (graphs, streams, bad pages)."""
import math

import numpy as np
import pytest
import torch

import serving_util as U

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _case(lengths, hq, hkv, d, x, cache, page, seed=0, gain=1.5):
    """CPU tensors of a call; the slots no row may read hold NaN."""
    g = torch.Generator().manual_seed(seed)
    table, total = U.pages(lengths, page, np.random.default_rng(seed))
    shape = (total, hkv, page, d)
    unit = 40.0 if cache == E4M3 else 1.0
    kc, vc = ((torch.randn(shape, generator=g) * unit).to(cache) for _ in range(2))
    ks = vs = None
    if cache == E4M3:
        ks, vs = (torch.rand(hkv, generator=g) * 0.02 + 0.015 for _ in range(2))
    live = torch.zeros((total, page), dtype=torch.bool)
    for b, n in enumerate(lengths):
        for p in range(n):
            live[int(table[b, p // page]), p % page] = True
    dead = (~live)[:, None, :, None].expand(shape)
    for c in (kc, vc):
        if cache == E4M3:
            c.view(torch.uint8)[dead] = 0x7F
        else:
            c[dead] = float("nan")
    q = (torch.randn((len(lengths), hq, d), generator=g) * gain).to(x)
    return dict(q=q, k_cache=kc, v_cache=vc, table=table, lengths=torch.tensor(lengths, dtype=torch.int32), k_scale=ks, v_scale=vs)


def _dev(c):
    return {k: None if v is None else v.cuda() for k, v in c.items()}


def _rows(c, rows):
    return {k: (v[rows] if k in ("q", "lengths", "table") else v) for k, v in c.items()}


def _but(c, length):
    return dict(c, lengths=torch.full_like(c["lengths"], length))


def _check(c, out, lse, scale=None, window=0, what="attention"):
    d = c["q"].shape[2]
    want, wlse, err, lerr = U.attention(c["q"], c["k_cache"], c["v_cache"], c["table"], c["lengths"],
                                        d ** -0.5 if scale is None else scale, window, c["k_scale"], c["v_scale"])
    U.assert_within(out, want, U.half_step(c["q"].dtype, want) + err, what + " out")
    U.assert_within(lse, wlse, lerr, what + " lse")


def _run(c, **kw):
    dev = _dev(c)
    lse = torch.full(c["q"].shape[:2], 7.0, device="cuda")
    out = mk.paged_attention(**dev, lse=lse, **kw)
    torch.cuda.synchronize()
    return out, lse


RAGGED = [0, 1, 2, 15, 16, 17, 31, 32, 33, 100, 257]


@pytest.mark.parametrize("x", [BF16, F32])
@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("hq,hkv,d", [(16, 8, 128), (8, 2, 64), (1, 1, 128), (3, 3, 64), (5, 1, 64), (16, 2, 128), (9, 1, 128),
                                      (32, 2, 64), (20, 1, 128), (33, 1, 64)])
def test_types_and_heads(x, cache, hq, hkv, d):
    c = _case(RAGGED, hq, hkv, d, x, cache, 16)
    _check(c, *_run(c))


@pytest.mark.parametrize("page", [1, 3, 8, 24, 100, 512])
@pytest.mark.parametrize("cache,d", [(BF16, 128), (BF16, 64), (E4M3, 128), (E4M3, 64)])
def test_page_sizes(page, cache, d):
    c = _case([1, 7, 0, 65, 130], 4, 2, d, BF16, cache, page, seed=1)
    _check(c, *_run(c))


@pytest.mark.parametrize("window", [1, 5, 16, 40, 1000])
@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_window(window, cache):
    c = _case(RAGGED, 8, 2, 64, F32, cache, 24, seed=2)
    _check(c, *_run(c, window=window), window=window)


@pytest.mark.parametrize("x,cache,hq,hkv,lengths", [
    (F32, BF16, 16, 8, [5119]),                     # one row: a cluster of CTAs for each kv head
    (F32, BF16, 2, 1, [20011]),                     # and a single one, of one kv head
    (BF16, BF16, 16, 8, [3000, 1, 0, 777, 2049]),
    (BF16, E4M3, 8, 2, [9001, 40]),
    (F32, E4M3, 12, 1, [4097, 4096, 4095]),         # more than 8 query heads a kv head
    (F32, BF16, 16, 1, [2000, 31]),                 # and the largest states in registers
])
def test_rows_joined_over_ctas(x, cache, hq, hkv, lengths):
    c = _case(lengths, hq, hkv, 128, x, cache, 16, seed=3)
    _check(c, *_run(c))


@pytest.mark.parametrize("n", [255, 257, 700])
def test_more_rows_than_threads(n):
    rng = np.random.default_rng(n)
    lengths = [int(v) for v in rng.integers(0, 40, n)]
    lengths[:3] = [0, 0, 0]
    c = _case(lengths, 2, 1, 64, BF16, BF16, 16, seed=4)
    _check(c, *_run(c))


def test_scale_and_large_scores():
    c = _case([200, 3, 64], 4, 2, 64, F32, BF16, 16, seed=5, gain=30.0)
    for scale in (0.02, 1.0, -0.5, 0.0):
        _check(c, *_run(c, scale=scale), scale=scale, what="scale %g" % scale)


@pytest.mark.parametrize("mag", [2.0 ** -100, 2.0 ** -20, 2.0 ** 60])
def test_query_magnitudes_with_an_8_bit_cache(mag):
    # the query is brought into fp16's range by a power of two: results do not depend on its size
    c = _case([70, 5], 4, 2, 128, F32, E4M3, 16, seed=6)
    small, _ = _run(c)
    c["q"] = c["q"] * mag
    big, _ = _run(c, scale=128 ** -0.5 / mag)
    assert torch.equal(small, big)


def test_padding_rows_are_left_as_they_were():
    c = _case([33, 0, 20], 4, 2, 64, BF16, BF16, 16, seed=7)
    c["lengths"] = torch.tensor([33, -1, 20], dtype=torch.int32)
    out, lse = torch.full((3, 4, 64), 5.0, device="cuda", dtype=BF16), torch.full((3, 4), 5.0, device="cuda")
    c["table"][1] = 2 ** 31 - 1                     # never looked at
    mk.paged_attention(**_dev(c), out=out, lse=lse)
    assert (out[1] == 5).all() and (lse[1] == 5).all()
    c["lengths"][1] = 0
    out[1], lse[1] = 0, -math.inf
    _check(c, out, lse)


def test_empty_calls():
    c = _dev(_case([0, 0], 4, 2, 64, BF16, BF16, 16))
    lse = torch.zeros((2, 4), device="cuda")
    assert (mk.paged_attention(**c, lse=lse) == 0).all() and (lse == -math.inf).all()
    none = dict(c, q=c["q"][:0], lengths=c["lengths"][:0])
    assert mk.paged_attention(**none).shape == (0, 4, 64)
    for t in (c["table"][:, :0], c["table"][:0, :0]):              # no pages, no rows
        r = t.shape[0]
        assert (mk.paged_attention(**dict(c, q=c["q"][:r], lengths=c["lengths"][:r], table=t)) == 0).all()


def test_strides_and_layouts():
    # pages of [slot][head][d], keys and values in one tensor, q a slice of a stacked projection, out of a wider one
    c = _case([100, 17, 250], 4, 2, 64, BF16, BF16, 24, seed=8)
    total = c["k_cache"].shape[0]
    kv = torch.zeros((total, 2, 24, 2, 64), dtype=BF16, device="cuda")
    kv[:, 0], kv[:, 1] = c["k_cache"].cuda().transpose(1, 2), c["v_cache"].cuda().transpose(1, 2)
    qkv = torch.zeros((3, 8, 64), dtype=BF16, device="cuda")
    qkv[:, 2:6] = c["q"].cuda()
    wide = torch.full((3, 5, 72), 9.0, dtype=BF16, device="cuda")
    table = torch.full((3, 40), -7, dtype=torch.int32, device="cuda")
    table[:, :c["table"].shape[1]] = c["table"].cuda()
    lse = torch.zeros((3, 4), device="cuda")
    out = mk.paged_attention(qkv[:, 2:6], kv[:, 0].transpose(1, 2), kv[:, 1].transpose(1, 2), table, c["lengths"].cuda(),
                             out=wide[:, 1:, :64], lse=lse)
    _check(c, out, lse)
    assert (wide[:, 0] == 9).all() and (wide[:, :, 64:] == 9).all()


def test_drafted_tokens_share_a_sequence():
    # four new tokens of one sequence: the same pages, growing lengths; the result overwrites the queries
    c = _case([103], 4, 2, 128, F32, BF16, 16, seed=9)
    q = torch.randn((4, 4, 128), generator=torch.Generator().manual_seed(1))
    lengths = torch.tensor([100, 101, 102, 103], dtype=torch.int32)
    lse = torch.zeros((4, 4), device="cuda")
    dev = q.cuda()
    out = mk.paged_attention(dev, c["k_cache"].cuda(), c["v_cache"].cuda(), c["table"].cuda().expand(4, -1), lengths.cuda(), out=dev, lse=lse)
    full = dict(c, q=q, lengths=lengths, table=c["table"].expand(4, -1))
    _check(full, out, lse)


def test_results_over_the_queries_of_long_rows():
    # rows cut over CTAs: no share of a row may see another's result in its query
    c = _case([5000, 4000, 7], 16, 8, 128, BF16, BF16, 16, seed=16)
    dev = _dev(c)
    want = mk.paged_attention(**dev)
    assert torch.equal(mk.paged_attention(**dev, out=dev["q"]), want)


def test_infinite_and_nan_scores():
    c = _case([40, 40], 2, 1, 64, F32, BF16, 16, seed=10)
    c["k_cache"][int(c["table"][0, 0]), 0, 3] = float("nan")       # one key of row 0
    out, lse = _run(c)
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    assert torch.isfinite(out[1]).all() and torch.isfinite(lse[1]).all()
    c["v_cache"][int(c["table"][1, 1]), 0, 2, 5] = float("inf")    # one value of row 1
    out, _ = _run(c)
    assert (out[1, :, 5] == math.inf).all() and torch.isfinite(out[1, :, :5]).all()
    # a key that scores -inf has no weight
    c = _case([40], 1, 1, 64, F32, BF16, 16, seed=17)
    c["q"][0, 0, 9] = -1.0
    want, wlse = _run(_but(c, 39))
    c["k_cache"][int(c["table"][0, 39 // 16]), 0, 39 % 16, 9] = float("inf")
    out, lse = _run(c)
    assert torch.equal(out, want) and torch.equal(lse, wlse)


@pytest.mark.parametrize("x", [BF16, F32])
def test_bad_pages_give_nan_and_a_status(x):
    c = _case([50, 50, 500, 20], 4, 2, 64, x, BF16, 16, seed=11)
    good = c["table"].clone()
    for bad in (-1, c["k_cache"].shape[0], 2 ** 31 - 1, -2 ** 31):
        c["table"] = good.clone()
        c["table"][0, 1] = bad
        c["table"][2, 20] = bad
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = _run(c, status=status)
        assert status.item() == -10
        with pytest.raises(mk.MKError):
            mk.check_status(status)
        assert torch.isnan(out[[0, 2]]).all() and torch.isnan(lse[[0, 2]]).all()
        _check(_rows(c, [1, 3]), out[[1, 3]], lse[[1, 3]])


def test_a_length_past_the_table():
    c = _case([50, 50], 4, 2, 64, BF16, BF16, 16, seed=12)
    for length in (c["table"].shape[1] * 16 + 1, 2 ** 31 - 1):
        c["lengths"] = torch.tensor([length, 50], dtype=torch.int32)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = _run(c, status=status)
        assert status.item() == -10 and torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
        _check(_rows(c, [1]), out[1:], lse[1:])
    ok = torch.zeros(1, dtype=torch.int32, device="cuda")
    c["lengths"][0] = 50
    _run(c, status=ok)
    mk.check_status(ok)


def test_same_bits_every_time_and_on_every_stream():
    c = _dev(_case([3000, 5, 777, 2049, 0], 16, 8, 128, BF16, BF16, 16, seed=13))
    lse = torch.empty((5, 16), device="cuda")
    want = mk.paged_attention(**c, lse=lse)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for i in range(12):                                            # calls that overlap, each with a workspace of its own
        l = torch.empty_like(lse)
        got.append((mk.paged_attention(**c, lse=l, stream=streams[i % 3]), l))
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want) and torch.equal(l, lse)


def test_captured_calls_follow_the_lengths():
    # two graphs over the same cache, replayed at once on two streams, with lengths that change between replays
    c = _dev(_case([2500, 900, 64], 16, 8, 128, BF16, BF16, 16, seed=14))
    lengths = [c["lengths"].clone() for _ in range(2)]
    graphs, outs = [], []
    mk.paged_attention(**c)
    torch.cuda.synchronize()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(mk.paged_attention(**dict(c, lengths=lengths[i])))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for a, b in (([2500, 900, 64], [1, 0, 7]), ([17, 17, 17], [2500, 3, 33]), ([0, 0, 0], [2499, 899, 63])):
        for i, n in enumerate((a, b)):
            lengths[i].copy_(torch.tensor(n, dtype=torch.int32))
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], mk.paged_attention(**dict(c, lengths=lengths[i])))


def test_offsets_past_32_bits():
    # a cache of more than 2^32 elements: the last pages start beyond it
    hkv, d, page = 8, 128, 64
    total = (1 << 32) // (hkv * page * d) + 4096
    kc = torch.empty((total, hkv, page, d), dtype=E4M3, device="cuda")
    vc = torch.empty_like(kc)
    c = _case([150], 16, hkv, d, BF16, E4M3, page, seed=15)
    use = [total - 1, 3, total - 2]
    for i, p in enumerate(use):
        for to, src in ((kc, c["k_cache"]), (vc, c["v_cache"])):
            to[p].copy_(src[int(c["table"][0, i])])
    lse = torch.zeros((1, 16), device="cuda")
    out = mk.paged_attention(c["q"].cuda(), kc, vc, torch.tensor([use], dtype=torch.int32, device="cuda"), c["lengths"].cuda(),
                             k_scale=c["k_scale"].cuda(), v_scale=c["v_scale"].cuda(), lse=lse)
    _check(c, out, lse)


@pytest.mark.parametrize("hq,hkv", [(4, 1), (16, 8), (48, 16), (64, 64), (100, 100), (160, 160), (40, 2)])
@pytest.mark.parametrize("length", [0, 1, 16, 300, 4000])
def test_one_row(hq, hkv, length):
    # one sequence: clusters of CTAs for each kv head, of every size, and more heads than there are clusters for
    c = _case([length], hq, hkv, 128, BF16, BF16, 16, seed=length + hq)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _check(c, *_run(c, status=status))
    mk.check_status(status)
    wide = dict(c, table=torch.cat([c["table"], torch.full((1, 600), 2 ** 30, dtype=torch.int32)], 1))
    _check(c, *_run(wide, status=status))                   # a table for more tokens than there are
    mk.check_status(status)
    if length:
        wide["table"][0, (length - 1) // 16] = -3
        out, lse = _run(wide, status=status)
        assert status.item() == -10 and torch.isnan(out).all() and torch.isnan(lse).all()


def test_one_row_left_alone_and_past_the_table():
    c = _case([40], 4, 2, 64, F32, E4M3, 8, seed=18)
    out, lse = torch.full((1, 4, 64), 5.0, device="cuda"), torch.full((1, 4), 5.0, device="cuda")
    c["lengths"][0] = -1
    mk.paged_attention(**_dev(c), out=out, lse=lse)
    assert (out == 5).all() and (lse == 5).all()
    c["lengths"][0] = 41
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mk.paged_attention(**_dev(c), out=out, lse=lse, status=status)
    assert status.item() == -10 and torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("x,cache", [(BF16, BF16), (F32, E4M3)])
def test_wide_tables_of_short_rows(window, x, cache):
    # the same rows by a table that fits them (rows kept whole) and by a wide one (rows cut where they fall)
    lengths = [int(v) for v in np.random.default_rng(5).integers(0, 700, 60)]
    c = _case(lengths, 8, 4, 64, x, cache, 24, seed=19)
    want = _run(c, window=window)
    _check(c, *want, window=window)
    wide = dict(c, table=torch.cat([c["table"], torch.full((60, 900), -1, dtype=torch.int32)], 1))
    _check(c, *_run(wide, window=window), window=window)


def test_a_workspace_is_asked_for_where_it_is_needed():
    import ctypes as C
    B = mk._binding
    lib = B.load_library()
    asked, held = [], []

    def give(context, n):
        asked.append(n)
        held.append(torch.empty(n, dtype=torch.uint8, device="cuda"))
        return held[-1].data_ptr()
    give, refuse = B.WORKSPACE_FN(give), B.WORKSPACE_FN(lambda context, n: None)
    hq, hkv, d, page = 4, 2, 64, 16
    g = torch.Generator().manual_seed(0)
    kc, vc = (torch.randn((300, hkv, page, d), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    # rows of up to 64 tiles of 32 slots (heads of 64) are not cut: 100 pages are 50 tiles, 300 are 150
    for rows, cols, needed in ((1, 300, 0), (3, 20, 0), (3, 100, 0), (3, 300, 1)):
        table = torch.arange(rows * cols, dtype=torch.int32, device="cuda").view(rows, cols) % 300
        lengths = torch.full((rows,), cols * page - 5, dtype=torch.int32, device="cuda")
        q = torch.randn((rows, hq, d), generator=g).cuda()
        want = mk.paged_attention(q, kc, vc, table, lengths)
        out = torch.zeros_like(q)
        kv = mk.serving.paged_struct(kc, vc, table)
        a = B.mk_attention_args.from_buffer_copy(mk.serving.native().check_attention(q, kc, vc, table, lengths, out=out))
        asked.clear()
        stream = torch.cuda.current_stream().cuda_stream
        assert lib.mk_paged_attention_ask(C.byref(kv), C.byref(a), give, None, stream) == 0
        torch.cuda.synchronize()
        assert torch.equal(out, want) and asked == [lib.mk_paged_attention_workspace(hq, hkv, d)] * needed
        out.zero_()
        assert lib.mk_paged_attention_ask(C.byref(kv), C.byref(a), refuse, None, stream) == (-8 if needed else 0)
        torch.cuda.synchronize()
        assert torch.equal(out, torch.zeros_like(q) if needed else want)   # refused before anything is enqueued
