"""``paged_append`` against its definition in 64 bits: norms, rotations, types,
strides, pages, padding, and that nothing else of the cache changes."""
import numpy as np
import pytest
import torch

import serving_util as U

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
EPS = 1e-6


def _bits(t):
    return t.view(torch.uint8 if t.dtype == E4M3 else torch.int16)


def _run(x, cache, hq, hkv, d, seqs, slots, page, norm=True, rope=None, interleaved=False, positions=None, seed=0, gain=1.0,
         layout=None, status=None, table_edit=None, inplace=False):
    """One call on seeded inputs; checks q_out and the whole cache. ``rope``: None, "slots", "positions" or sections."""
    g = torch.Generator().manual_seed(seed)
    n = len(slots)
    lengths = [0] * (max(list(seqs), default=0) + 1)
    for s, p in zip(seqs, slots):
        lengths[s] = max(lengths[s], p + 1)
    table, total = U.pages(lengths, page, np.random.default_rng(seed))
    unit = 30.0 if cache == E4M3 else 1.0
    kc, vc = ((torch.randn((total, hkv, page, d), generator=g) * unit).to(cache) for _ in range(2))
    qkv = (torch.randn((n, hq + 2 * hkv, d), generator=g) * gain).to(x)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    ks = vs = None
    if cache == E4M3:
        ks, vs = (torch.rand(hkv, generator=g) * 0.02 + 0.01 for _ in range(2))
    qn, kn = ((1 + 0.1 * torch.randn(d, generator=g)).to(BF16) for _ in range(2)) if norm else (None, None)
    rows = 3 * max(list(slots), default=0) + 16
    sections = rope if isinstance(rope, tuple) else None
    pos = torch.tensor(slots).clamp_min(0)
    if rope == "positions":
        pos = pos * 2 + 1
    if sections:
        pos = torch.stack([pos, pos + 7, 2 * pos + 3])
    if positions is not None:
        pos = positions
    if table_edit:
        table_edit(table, total)

    # the definition
    angle = None
    if rope:
        angle = U.rotary(pos, d)
        if sections:
            st = U.pair_streams(d, sections, interleaved)
            angle = torch.stack([angle[st[i], :, i] for i in range(d // 2)], -1)
    wq, eq = U.turned(q, qn, angle, EPS)
    wk, ek = U.turned(k, kn, angle, EPS)
    wv, ev = U.turned(v, None, None, EPS)
    if cache == E4M3:
        kd64, vd64 = ks.to(U.F64)[:, None], vs.to(U.F64)[:, None]
        wk, ek = wk / kd64, ek / kd64 + (wk / kd64).abs() * 2.0 ** -23
        wv = wv / vd64
        ev = wv.abs() * 2.0 ** -22
        wk, wv = wk.clamp(-448, 448), wv.clamp(-448, 448)
    held = [kc.to(U.F64), vc.to(U.F64)]
    tol = [torch.zeros_like(held[0]) for _ in range(2)]
    done = torch.zeros(n, dtype=torch.bool)
    for i, (s, p) in enumerate(zip(seqs, slots)):
        if p < 0 or p // page >= table.shape[1] or not 0 <= int(table[s, p // page]) < total:
            continue
        if rope and not (0 <= int(pos[..., i].min()) and int(pos[..., i].max()) < rows):
            continue
        done[i] = True
        to = int(table[s, p // page]), slice(None), p % page
        for c, (val, err) in enumerate(((wk, ek), (wv, ev))):
            held[c][to] = val[i]
            # a value just below a power of two may round up past it: its step is taken at value + error
            tol[c][to] = U.half_step(cache, val[i].abs() + err[i]) + err[i]

    # the call
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    kd, vd = dev(kc), dev(vc)
    if layout:                                       # [page][slot][head][d], keys and values in one tensor
        kv = torch.empty((total, 2, page, hkv, d), dtype=cache, device="cuda")
        _bits(kv)[:, 0], _bits(kv)[:, 1] = _bits(kd).transpose(1, 2), _bits(vd).transpose(1, 2)
        kd, vd = kv[:, 0].transpose(1, 2), kv[:, 1].transpose(1, 2)
    qd = qkv.cuda()
    mine = list(range(n)) == list(seqs)
    q_in = qd[:, :hq]
    q_out = q_in if inplace else torch.full((n, hq, d), 3.0, dtype=x, device="cuda")
    before = q_out.clone()
    give = rope and (rope != "slots" or positions is not None)
    out = mk.paged_append(qd[:, hq:hq + hkv], qd[:, hq + hkv:], kd, vd, dev(table), torch.tensor(slots, dtype=torch.int32).cuda(),
                          seqs=None if mine else torch.tensor(seqs, dtype=torch.int32).cuda(), q=q_in if hq else None,
                          q_out=q_out if hq else None, rope=mk.rope_table(rows, d) if rope else None,
                          positions=dev(pos.to(torch.int32).contiguous()) if give else None,
                          mrope_sections=sections, mrope_interleaved=interleaved, q_norm=dev(qn), k_norm=dev(kn), eps=EPS,
                          k_scale=dev(ks), v_scale=dev(vs), status=status)
    torch.cuda.synchronize()
    if hq:
        d_ = done.cuda()
        U.assert_within(out[d_], wq[done], (U.half_step(x, wq.abs() + eq) + eq)[done], "q_out")
        assert torch.equal(out[~d_], before[~d_])
    for name, got, want, t in (("keys", kd, held[0], tol[0]), ("values", vd, held[1], tol[1])):
        U.assert_within(got, want, t, name)
    if not inplace:
        assert torch.equal(qd.cpu(), qkv)


@pytest.mark.parametrize("x", [BF16, F32])
@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("hq,hkv,d", [(16, 8, 128), (8, 2, 64), (3, 1, 64), (0, 2, 128), (5, 5, 128)])
@pytest.mark.parametrize("norm", [True, False])
def test_decode_rows(x, cache, hq, hkv, d, norm):
    _run(x, cache, hq, hkv, d, range(7), [0, 15, 16, 17, 100, 255, 31], 16, norm=norm, rope="slots")


@pytest.mark.parametrize("rope,interleaved", [(None, False), ("positions", False), ((24, 20, 20), False), ((24, 20, 20), True)])
@pytest.mark.parametrize("x", [BF16, F32])
def test_rotations(rope, interleaved, x):
    _run(x, BF16, 16, 8, 128, range(3), [300, 4, 0], 16, rope=rope, interleaved=interleaved, seed=1)


@pytest.mark.parametrize("page", [1, 5, 24, 64])
@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_prompts(page, cache):
    # three prompts in one call, one of a single token, rows of a sequence out of order
    seqs = [2] * 50 + [0] + [1] * 33
    slots = list(range(49, -1, -1)) + [0] + list(range(33))
    _run(BF16, cache, 4, 2, 64, seqs, slots, page, rope="slots", seed=2)


def test_one_row_and_many():
    _run(F32, BF16, 16, 8, 128, [0], [300], 16, rope=(24, 20, 20), seed=3)
    _run(BF16, E4M3, 2, 1, 64, [0] * 3001, list(range(3001)), 100, rope="slots", seed=4)


def test_layouts_and_in_place_queries():
    _run(BF16, BF16, 4, 2, 64, range(4), [3, 30, 11, 0], 12, rope="slots", seed=5, layout="nhd")
    _run(F32, E4M3, 4, 2, 128, range(4), [3, 30, 11, 0], 12, rope="slots", seed=6, layout="nhd", inplace=True)


def test_padding_rows_are_left_alone():
    _run(BF16, BF16, 4, 2, 64, range(5), [3, -1, 7, -1, -2 ** 31], 16, rope="slots", seed=7)


def test_values_that_saturate():
    _run(F32, E4M3, 2, 2, 64, range(3), [1, 2, 3], 16, norm=False, rope="slots", seed=8, gain=40.0)


def test_special_values_in_an_8_bit_cache():
    k = torch.zeros((1, 1, 64), device="cuda")
    k[0, 0, :5] = torch.tensor([float("inf"), -float("inf"), float("nan"), 449.0, 2.0 ** -10])
    kc = torch.zeros((1, 1, 4, 64), dtype=E4M3, device="cuda")
    vc = torch.zeros_like(kc)
    mk.paged_append(k, k, kc, vc, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.tensor([2], dtype=torch.int32, device="cuda"))
    for c in (kc, vc):
        got = c[0, 0, 2, :5].float().tolist()
        assert got[:2] == [448.0, -448.0] and got[2] != got[2] and got[3] == 448.0 and got[4] == 0.0   # a tie goes to even


@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_bad_pages_are_reported_and_skipped(cache):
    def edit(table, total):
        table[0, 1], table[2, 0] = total, -5
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _run(BF16, cache, 4, 2, 64, range(4), [20, 20, 3, 9], 16, rope="slots", seed=9, status=status, table_edit=edit)
    assert status.item() == -10


def test_sequences_and_slots_outside_the_table():
    kc = torch.ones((2, 1, 4, 64), dtype=BF16, device="cuda")
    vc = kc.clone()
    k = torch.zeros((4, 1, 64), dtype=BF16, device="cuda")
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    status = i32(0)
    mk.paged_append(k, k, kc, vc, table, i32(1, 8, 2 ** 31 - 1, 0), seqs=i32(1, 0, 0, -1), status=status)
    assert status.item() == -10 and (kc == 1).all() and (vc == 1).all()


def test_positions_outside_the_rotary_table():
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos = torch.tensor([5, 31, 10 ** 6, -1])               # the table has 3 * 5 + 16 = 31 rows
    _run(BF16, BF16, 4, 2, 64, range(4), [5, 3, 2, 1], 16, rope="positions", seed=10, status=status, positions=pos)
    assert status.item() == -9
    pos = torch.tensor([[5, 31, 4], [5, 4, 4], [5, 4, 31]])
    _run(BF16, BF16, 4, 2, 64, range(3), [5, 3, 2], 16, rope=(12, 10, 10), seed=11, positions=pos)


def test_captured_and_replayed():
    g0 = torch.Generator().manual_seed(0)
    kc, vc = (torch.zeros((8, 2, 16, 64), dtype=BF16, device="cuda") for _ in range(2))
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    slots = torch.tensor([3, 4], dtype=torch.int32, device="cuda")
    k, v, q = (torch.randn((2, 2, 64), generator=g0).to(BF16).cuda() for _ in range(3))
    rope = mk.rope_table(64, 64)
    graph = torch.cuda.CUDAGraph()
    mk.paged_append(k, v, kc, vc, table, slots, q=q, rope=rope)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        q_out = mk.paged_append(k, v, kc, vc, table, slots, q=q, rope=rope)
    for at in ((0, 63), (40, 17), (-1, 5)):
        kc.zero_(), vc.zero_(), q_out.zero_()
        slots.copy_(torch.tensor(at, dtype=torch.int32))
        k.copy_(torch.randn((2, 2, 64), generator=g0))
        graph.replay()
        k2, v2, q2 = torch.zeros_like(kc), torch.zeros_like(vc), torch.zeros_like(q)
        mk.paged_append(k, v, k2, v2, table, slots, q=q, q_out=q2, rope=rope)
        torch.cuda.synchronize()
        assert torch.equal(kc, k2) and torch.equal(vc, v2) and torch.equal(q_out, q2)


# Token counts past which persistent warps take the tokens (a thread for every part of every head would no longer be
# resident): heads in whole and broken groups of 4, rows without queries, more tokens than a warp looks up at once.
@pytest.mark.parametrize("x,cache,hq,hkv,d,n,rope,interleaved,norm", [
    (BF16, E4M3, 16, 8, 128, 700, "slots", False, True),
    (F32, BF16, 16, 8, 128, 300, (24, 20, 20), True, True),
    (BF16, BF16, 9, 3, 64, 2100, (12, 10, 10), False, True),
    (F32, E4M3, 5, 5, 64, 1100, "positions", False, False),
    (BF16, BF16, 0, 2, 128, 3800, None, False, True),
    (F32, E4M3, 33, 1, 128, 250, None, False, False),
    (BF16, E4M3, 64, 64, 128, 120, "slots", False, False),
    (BF16, BF16, 2, 1, 64, 59000, "slots", False, True)])
def test_many_tokens(x, cache, hq, hkv, d, n, rope, interleaved, norm):
    seqs = [i % 3 for i in range(n)]
    slots = [i // 3 for i in range(n)]
    for i in (5, 77, n - 1):
        slots[i] = -1
    _run(x, cache, hq, hkv, d, seqs, slots, 20, norm=norm, rope=rope, interleaved=interleaved, seed=12)


@pytest.mark.parametrize("layout", [None, "nhd"])
def test_many_tokens_and_some_that_are_refused(layout):
    n = 600
    seqs = [i % 3 for i in range(n)]
    slots = [i // 3 for i in range(n)]
    pos = torch.tensor(slots)
    pos[40], pos[333] = 10 ** 6, -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def edit(table, total):
        table[0, 1], table[2, 0] = total, -5
    _run(BF16, E4M3, 24, 4, 128, seqs, slots, 16, rope="positions", seed=13, status=status, positions=pos, table_edit=edit,
         layout=layout, inplace=layout is not None)
    assert status.item() in (-9, -10)


def test_many_tokens_captured_and_replayed():
    g0 = torch.Generator().manual_seed(0)
    n = 1000
    kc, vc = (torch.zeros((70, 8, 16, 128), dtype=BF16, device="cuda") for _ in range(2))
    table = torch.arange(70, dtype=torch.int32, device="cuda").view(1, 70)
    slots, seqs = (torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(2))
    q, k, v = (torch.randn((n, h, 128), generator=g0).to(BF16).cuda() for h in (16, 8, 8))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q_out = mk.paged_append(k, v, kc, vc, table, slots, seqs=seqs, q=q)
    order = torch.randperm(n, generator=g0).to(torch.int32)
    for _ in range(3):
        slots.copy_(order)
        graph.replay()
        torch.cuda.synchronize()
        at = order.long().cuda()
        for c, r in ((kc, k), (vc, v)):
            assert torch.equal(c[at // 16, :, at % 16], r)
        assert torch.equal(q_out, q)
        order = order.roll(1)
