"""How the operators of prompts and of a step's two ends are called: first calls in a capture, calls at once on
several streams, captured calls next to one another, errors on a side stream, autograd, results of one allocation."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_first_calls_inside_a_capture():
    # a new process whose first call of each operator is captured: nothing that a capture forbids happens there
    code = """
import torch
import persistent_transformer_megakernel_gb300 as mk
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
kc, vc = (torch.randn((300, 2, 16, 64), device="cuda").bfloat16() for _ in range(2))
kq, vq = (c.to(torch.float8_e4m3fn) for c in (kc, vc))
q = torch.randn((90, 4, 64), device="cuda").bfloat16()
table, long_table = torch.arange(300, dtype=torch.int32, device="cuda").view(2, 150), torch.zeros((2, 300), dtype=torch.int32, device="cuda")
lengths, counts, starts = i32([1000, 60]), i32([50, 30]), i32([0, 50, 80])
free, used = torch.arange(600, dtype=torch.int32, device="cuda"), i32([0])
x, w = torch.randn((90, 256), device="cuda").bfloat16(), torch.randn((300, 256), device="cuda")
many = torch.randn((600, 256), device="cuda").bfloat16()
wc, ws = mk.quantize_fp8_weight(w)
ids = torch.randint(0, 1000, (3, 40), dtype=torch.int32, device="cuda")
logits = torch.randn((3, 1000), device="cuda")
torch.cuda.synchronize()
def step():
    plan = mk.paged_plan(lengths, long_table, free, used, 16, counts=counts, rows=90)
    got = list(plan)
    for k, v in ((kc, vc), (kq, vq)):
        got.append(mk.paged_prompt_attention(q, k, v, table, starts, lengths, window=500, sinks=4)[:80])
        got.append(mk.paged_prompt_attention(q, k, v, table[:, :7], starts, i32_lengths)[:80])
        got.append(mk.paged_attention(q[:2], k, v, table, lengths, window=500, sinks=4))
    for a in (x, many):
        c, s = mk.quantize_fp8(a)
        got += [c.float(), s, mk.matmul_fp8(c, s, wc, ws)]
    got.append(mk.adjust_logits(logits, tokens=ids, repetition=ones * 2, frequency=ones, presence=ones))
    return got
ones, i32_lengths = torch.ones(3, device="cuda"), i32([100, 60])
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = step()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, step()))
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr


class Work:
    """Calls of all operators that need no other's results, on inputs of their own."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        normal = lambda *s: torch.randn(s, generator=g).cuda()
        self.kc, self.vc = (normal(200, 2, 16, 64).to(BF16) for _ in range(2))
        self.q = normal(700, 4, 64).to(BF16)
        self.table = torch.randperm(200, generator=g).int().cuda().view(1, 200)
        self.starts, self.lengths = i32([0, 700]), i32([3000])
        self.x, self.w = normal(40, 2048).to(BF16), mk.quantize_fp8_weight(normal(512, 2048))
        self.counts, self.used = torch.randint(0, 30, (500,), generator=g).int().cuda(), i32([3])
        self.free, self.len = torch.arange(9000).int().cuda(), torch.randint(0, 300, (500,), generator=g).int().cuda()
        self.pages = torch.zeros((500, 30), dtype=torch.int32, device="cuda")
        self.logits, self.ids = normal(4, 30000), torch.randint(0, 30000, (4, 900), generator=g).int().cuda()
        self.ones = torch.full((4,), 1.25, device="cuda")

    def run(self):
        out = [mk.paged_prompt_attention(self.q, self.kc, self.vc, self.table, self.starts, self.lengths)]
        c, s = mk.quantize_fp8(self.x)
        out += [c.view(torch.uint8), s, mk.matmul_fp8(c, s, *self.w)]
        out += list(mk.paged_plan(self.len, self.pages, self.free, self.used, 16, counts=self.counts, rows=20000)) + [self.pages]
        return out + [mk.adjust_logits(self.logits, tokens=self.ids, repetition=self.ones, presence=self.ones, frequency=self.ones)]


def test_calls_at_once_and_captured_calls_next_to_one_another():
    works = [Work(i) for i in range(3)]
    want = [[t.clone() for t in w.run()] for w in works]
    streams = [torch.cuda.Stream() for _ in works]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got = []
        for w, s in zip(works, streams):
            with torch.cuda.stream(s):
                got.append(w.run())
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    # graphs that are replayed at once on streams of their own
    graphs, outs = [], []
    for w in works:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(w.run())
        graphs.append(g)
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_results_of_one_allocation_are_apart():
    for n, rows in ((0, 0), (0, 5), (1, 1), (3, 7), (5, 4)):
        lengths, counts = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
        got = mk.paged_plan(lengths, torch.zeros((n, 2), dtype=torch.int32, device="cuda"), i32([4, 5, 6]), i32([0]), 16, counts=counts, rows=rows)
        assert [t.shape for t in got] == [(rows,), (rows,), (n + 1,), (n,), (1,)]
        for i, t in enumerate(got):
            assert t.is_contiguous() and t.dtype == torch.int32 and (t.numel() == 0 or t.data_ptr() % 16 == 0)
            t.fill_(i + 7)
        assert all((t == i + 7).all() for i, t in enumerate(got))
    for m, k in ((0, 128), (1, 16), (3, 144), (5, 128)):
        codes, scales = mk.quantize_fp8(torch.ones((m, k), dtype=BF16, device="cuda"))
        assert codes.shape == (m, k) and codes.dtype == E4M3 and scales.shape == (m, -(-k // 128)) and scales.dtype == torch.float32
        scales.fill_(3.0)
        assert (codes.float() == 448).all()
        codes.view(torch.uint8).fill_(0)
        assert (scales == 3).all()


def test_an_error_on_a_side_stream():
    kc, vc = (torch.zeros((2, 1, 4, 64), dtype=BF16, device="cuda") for _ in range(2))
    table = torch.full((1, 2), 99, dtype=torch.int32, device="cuda")                # a page that is none
    q = torch.ones((3, 1, 64), dtype=BF16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    starts, lengths = i32([0, 3]), i32([5])
    torch.cuda.synchronize()
    mk.paged_prompt_attention(q, kc, vc, table, starts, lengths, status=status, stream=side)
    with pytest.raises(mk.MKError) as e:
        mk.check_status(status, stream=side)
    assert e.value.code == -10
    status.zero_()
    torch.cuda.synchronize()
    plan = mk.paged_plan(lengths, table, i32([1]), i32([1]), 4, counts=i32([4]), rows=4, status=status, stream=side)
    with pytest.raises(mk.MKError) as e:
        mk.check_status(status, stream=side)
    assert e.value.code == -3 and plan[4].item() == 1


def test_what_is_written_counts_as_changed_and_no_gradients():
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros((2, 1, 16, 64), dtype=BF16, device="cuda") for _ in range(2))
    q, one, status = torch.ones((3, 1, 64), dtype=BF16, device="cuda"), i32([3]), z(1)
    table, free = z(1, 2), i32([0, 1])

    def grown(written, read, f):
        before = [t._version for t in written + read]
        f()
        assert [t._version for t in written] == [v + 1 for v in before[:len(written)]]
        assert [t._version for t in read] == before[len(written):]

    outs = dict(seqs=z(3), slots=z(3), starts=z(2), totals=z(1), used_out=z(1))
    grown((table, status, *outs.values()), (one, free), lambda: mk.paged_plan(z(1), table, free, z(1), 16, counts=one, rows=3, status=status, **outs))
    out, lse = torch.zeros_like(q), torch.zeros((3, 1), device="cuda")
    grown((out, lse, status), (q, kc, vc, one), lambda: mk.paged_prompt_attention(q, kc, vc, table, i32([0, 3]), one, out=out, lse=lse, status=status))
    x, codes, scales = torch.ones((3, 128), dtype=BF16, device="cuda"), torch.zeros((3, 128), dtype=E4M3, device="cuda"), torch.zeros((3, 1), device="cuda")
    grown((codes, scales), (x,), lambda: mk.quantize_fp8(x, codes=codes, scales=scales))
    w, ws = mk.quantize_fp8_weight(torch.ones((8, 128), device="cuda"))
    y = torch.zeros((3, 8), dtype=torch.float32, device="cuda")
    grown((y,), (codes, scales, w, ws), lambda: mk.matmul_fp8(codes, scales, w, ws, out=y))
    grown((y,), (w, ws), lambda: mk.adjust_logits(y, bias_ids=z(3, 1), bias=torch.ones((3, 1), device="cuda"), out=y))
    # there is no backward: what requires gradients is refused while they are recorded
    for t, f in ((q, lambda a: mk.paged_prompt_attention(a, kc, vc, table, i32([0, 3]), one)), (x, mk.quantize_fp8),
                 (scales, lambda a: mk.matmul_fp8(codes, a, w, ws)), (y, mk.adjust_logits)):
        leaf = t.clone().requires_grad_()
        with pytest.raises(ValueError, match="gradient"):
            f(leaf)
        with torch.no_grad():
            f(leaf)


def test_more_than_2_to_the_31_elements():
    # an input, a result and rows of logits that a 32-bit index does not reach, at rows before and behind that border
    g = torch.Generator(device="cuda").manual_seed(5)
    m, k = (1 << 31) // 2048 + 300, 2048
    rows = [0, 1, (1 << 31) // k - 1, (1 << 31) // k, (1 << 31) // k + 1, m - 1]
    x = torch.zeros((m, k), dtype=BF16, device="cuda")
    x[rows] = torch.randn((len(rows), k), generator=g, device="cuda").to(BF16)
    codes, scales = mk.quantize_fp8(x)
    want, want_scales = mk.quantize_fp8(x[rows])
    assert torch.equal(codes.view(torch.uint8)[rows], want.view(torch.uint8)) and torch.equal(scales[rows], want_scales)
    assert not codes.view(torch.uint8)[2:500].any() and (scales[2:500] == 1).all()   # (a block of zeros)
    w, ws = mk.quantize_fp8_weight(torch.randn((2056, 2048), generator=g, device="cuda"))
    few = mk.matmul_fp8(want, want_scales, w, ws, dtype=torch.float32)
    big = mk.matmul_fp8(codes, scales, w, ws, dtype=torch.float32)     # 8.6 GB and more
    # (sums of few tiles are shared by CTAs: another order, at most 2048 / 128 partial sums of 128 terms)
    bound = (want.float().abs() * want_scales.repeat_interleave(128, 1)) @ (w.float().abs() * ws.repeat_interleave(128, 1)[torch.arange(2056, device="cuda") // 128]).t()
    assert ((big[rows] - few).abs() <= 40 * 2.0 ** -23 * bound + 1e-30).all() and not big[2:500].any()
    # the same into a result whose rows are not on 16 bytes, where numbers leave one by one
    wide = torch.zeros((m, 2057), dtype=torch.float32, device="cuda")
    mk.matmul_fp8(codes, scales, w, ws, out=wide[:, :2056])
    assert torch.equal(wide[:, :2056][rows], big[rows]) and not wide[:, 2056].any()
    del x, codes, scales, big, wide
    n, v = (1 << 31) // 50000 + 5, 50000
    logits = torch.zeros((n, v), dtype=BF16, device="cuda")
    at = [0, 7, n - 6, n - 5, n - 1]
    logits[at] = torch.randn((len(at), v), generator=g, device="cuda").to(BF16)
    ids = torch.randint(0, v, (n, 30), generator=g, device="cuda", dtype=torch.int32)
    ones = torch.full((n,), 1.25, device="cuda")
    got = mk.adjust_logits(logits, tokens=ids, repetition=ones, presence=ones, frequency=ones)
    part = mk.adjust_logits(logits[at], tokens=ids[at], repetition=ones[:5], presence=ones[:5], frequency=ones[:5])
    assert torch.equal(got[at], part)


@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_in_place_where_rows_are_worked_on_again(cache):
    # values behind a row's own token that are no numbers, so that its first result is none either
    g = torch.Generator().manual_seed(11)
    kc, vc = (torch.randn((8, 2, 16, 64), generator=g).to(BF16) for _ in range(2))
    vc[5:] = float("nan")
    kc, vc = kc.to(cache).cuda(), vc.to(cache).cuda()
    q = torch.randn((100, 4, 64), generator=g).to(BF16).cuda()
    table, starts, lengths = torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8), i32([0, 100]), i32([128])
    want = mk.paged_prompt_attention(q, kc, vc, table, starts, lengths)
    assert torch.isfinite(want[:50]).all()
    got = q.clone()
    mk.paged_prompt_attention(got, kc, vc, table, starts, lengths, out=got)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("window", [0, 1500])
def test_few_sequences_and_the_same_among_many(cache, window):
    # the tasks of few sequences are found otherwise than those of many: empty ones behind them make many of few
    g = torch.Generator().manual_seed(21)
    kc, vc = (torch.randn((500, 2, 16, 64), generator=g).to(cache).cuda() for _ in range(2))
    for new, old in (([300, 40, 1, 0, 200], [1000, 3000, 5, 70, 0]), ([4], [7000]), ([1, 1, 1], [7000, 0, 2500]), ([900], [0]), ([2000, 30], [0, 4000])):
        lengths = [a + b for a, b in zip(new, old)]
        rows = sum(new)
        starts = [sum(new[:i]) for i in range(len(new) + 1)]
        table = torch.randint(0, 500, (len(new) + 40, 450), generator=g).int().cuda()
        q = torch.randn((rows, 4, 64), generator=g).to(BF16).cuda()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        few_lse, many_lse = (torch.full((rows, 4), -7.0, device="cuda") for _ in range(2))
        few = mk.paged_prompt_attention(q, kc, vc, table, i32(starts), i32(lengths), window=window, sinks=4, lse=few_lse, status=status)
        many = mk.paged_prompt_attention(q, kc, vc, table, i32(starts + [rows] * 40), i32(lengths + [9] * 40), window=window, sinks=4, lse=many_lse, status=status)
        mk.check_status(status)
        # weights and results are rounded to bf16 in both, each by 2^-8 at most, and a result is no larger than the largest value
        assert ((few.double() - many.double()).abs() <= 4 * 2.0 ** -8 * vc.float().abs().max()).all()
        # lse: tokens of a row summed in other parts, (64 + n / 32) 2^-23 each way, and 2^-22 of it for the logarithm
        assert ((few_lse.double() - many_lse.double()).abs() <= 2 * (64 + max(lengths) / 32) * 2.0 ** -23 + 2.0 ** -20 * many_lse.abs()).all()


def test_starts_that_decrease_among_long_contexts():
    g = torch.Generator().manual_seed(22)
    kc, vc = (torch.randn((400, 2, 16, 64), generator=g).to(BF16).cuda() for _ in range(2))
    table = torch.randint(0, 400, (5, 400), generator=g).int().cuda()
    q = torch.randn((400, 4, 64), generator=g).to(BF16).cuda()
    want = mk.paged_prompt_attention(q, kc, vc, table[:2], i32([0, 150, 300]), i32([5000, 3000]))
    for starts, lengths in (([0, 150, 300, 100, 80, 80], [5000, 3000, 900, 900, 900]), ([0, 150, 300, 500, 400, 380], [5000, 3000, 900, 900, 900]),
                            ([0, 150, 300, 300, 300, 300], [5000, 3000, -1, 7000, 2 ** 31 - 1])):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = mk.paged_prompt_attention(q, kc, vc, table, i32(starts), i32(lengths), status=status)
        # sequences are cut otherwise among others: as above
        assert ((got[:300].double() - want[:300].double()).abs() <= 4 * 2.0 ** -8 * vc.float().abs().max()).all()
        if starts[-1] < 300 or starts[3] > 400:
            with pytest.raises(mk.MKError):
                mk.check_status(status)
        else:
            mk.check_status(status)


def test_deterministic_mode_fills_new_results_and_changes_none():
    w = Work(9)
    want = [t.clone() for t in w.run()]
    kc, vc = (torch.randn((4, 1, 16, 64), device="cuda").to(BF16) for _ in range(2))
    q, table = torch.randn((5, 2, 64), device="cuda").to(BF16), torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    torch.use_deterministic_algorithms(True)
    try:
        got = w.run()
        out = mk.paged_prompt_attention(q, kc, vc, table, i32([0, 3]), i32([20]))    # two rows of no sequence
    finally:
        torch.use_deterministic_algorithms(False)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.isfinite(out[:3]).all() and torch.isnan(out[3:]).all()
