"""Refusals of the operators of prompts and of a step's two ends (no GPU)."""
import ctypes as C
import inspect
import os

import pytest
import torch

import prompt_util as P

import persistent_transformer_megakernel_gb300 as mk
from persistent_transformer_megakernel_gb300 import _binding as B
from persistent_transformer_megakernel_gb300 import serving as S

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn

if not os.path.exists(mk.lib_path()) or not os.path.exists(os.path.join(os.path.dirname(mk.lib_path()), "_mktorch.so")):
    from persistent_transformer_megakernel_gb300 import build
    build.build()


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def refused(f, *changes, error=ValueError):
    for kw in changes:
        with pytest.raises(error):
            f(**kw)


def _plan(**kw):
    a = dict(lengths=i32(3), table=i32(4, 5), free=i32(9), used=i32(1), page_size=16, counts=i32(3), rows=7)
    a.update(kw)
    return B.mk_plan_args.from_buffer_copy(S.native().check_plan(**a))


def test_plan_tensors():
    a = _plan()
    assert (a.n, a.rows, a.page_size, a.table_cols, a.table_stride, a.free_count) == (3, 7, 16, 5, 5, 9)
    assert _plan(counts=None, rows=None).rows == 3 and _plan(counts=None, rows=3).counts is None
    assert _plan(table=i32(3, 40)[:, 2:9]).table_stride == 40
    both = i32(3)
    assert _plan(lengths=both, totals=both).totals == both.data_ptr()
    one = i32(1)
    assert _plan(used=one, used_out=one).used_out == one.data_ptr()
    buf = i32(40)
    refused(_plan, dict(lengths=i32(3).long()), dict(lengths=i32(3, 1)), dict(table=i32(2, 5)), dict(table=i32(5, 4).t()), dict(table=i32(1, 5).expand(3, -1)),
            dict(table=i32(4, 5).long()), dict(free=i32(2, 2)), dict(free=i32(18)[::2]), dict(used=i32(2)), dict(used=None), dict(page_size=0), dict(page_size=-4),
            dict(counts=i32(4)), dict(counts=None, rows=4), dict(rows=-1), dict(seqs=i32(6)), dict(slots=i32(8)), dict(starts=i32(3)), dict(totals=i32(4)),
            dict(used_out=i32(2)), dict(status=i32(2)), dict(seqs=buf[:7], slots=buf[6:13]), dict(counts=buf[:3], totals=buf[2:5]),
            dict(lengths=buf[:3], seqs=buf[:7]), dict(table=buf[:20].view(4, 5), slots=buf[19:26]), dict(table=buf[:20].view(4, 5), free=buf[10:19]),
            dict(lengths=buf[:3], totals=buf[1:4]), dict(free=buf[:9], starts=buf[8:12]))
    refused(_plan, dict(page_size="x"), dict(rows=1.5), dict(nothing=1), error=TypeError)
    with pytest.raises(ValueError, match="CUDA"):
        mk.paged_plan(i32(3), i32(3, 2), i32(4), i32(1), 16)


CACHE = dict(k_cache=torch.zeros((6, 2, 16, 64), dtype=BF16), v_cache=torch.zeros((6, 2, 16, 64), dtype=BF16), table=i32(3, 4))


def _prompt(**kw):
    a = dict(CACHE, q=torch.zeros((9, 4, 64), dtype=BF16), starts=i32(4), lengths=i32(3), scale=None, window=0, sinks=0, out=torch.zeros((9, 4, 64), dtype=BF16),
             lse=torch.zeros((9, 4)), status=None)
    a.update(kw)
    return B.mk_prompt_args.from_buffer_copy(S.native().check_prompt(**a))


def test_prompt_tensors():
    a = _prompt()
    assert (a.n, a.rows, a.n_q_heads, a.scale, a.q_row) == (3, 9, 4, 0.125, 256)
    assert _prompt(starts=i32(2), lengths=i32(1)).n == 1
    assert (_prompt(window=2 ** 40).window, _prompt(sinks=2 ** 40).sinks) == (2 ** 31 - 1, 2 ** 31 - 1)
    q = torch.zeros((9, 4, 64), dtype=BF16)
    assert _prompt(q=q, out=q).out == q.data_ptr()
    refused(_prompt, dict(q=torch.zeros((9, 4, 64))), dict(q=torch.zeros((9, 4, 64), dtype=torch.float16)), dict(q=torch.zeros((9, 3, 64), dtype=BF16)),
            dict(q=torch.zeros((9, 4, 128), dtype=BF16)), dict(q=None), dict(starts=i32(3)), dict(starts=None), dict(starts=i32(4).long()), dict(lengths=None),
            dict(lengths=i32(4), starts=i32(5)), dict(lengths=i32(3, 1)), dict(window=-1), dict(sinks=-1), dict(scale=float("nan")), dict(scale=float("-inf")),
            dict(out=torch.zeros((9, 4, 64))), dict(out=torch.zeros((8, 4, 64), dtype=BF16)), dict(out=torch.zeros((1, 4, 64), dtype=BF16).expand(9, -1, -1)),
            dict(lse=torch.zeros((9, 4), dtype=BF16)), dict(lse=torch.zeros((4, 9)).t()), dict(out=CACHE["k_cache"].view(-1)[:2304].view(9, 4, 64)),
            dict(q=torch.zeros((9, 5, 64), dtype=BF16)[:, :4], out=torch.zeros(9 * 256 + 8, dtype=BF16)[4:-4].view(9, 4, 64)), dict(status=i32(2)))
    both = torch.zeros((18, 4, 64), dtype=BF16)
    refused(_prompt, dict(q=both[:9], out=both[8:17]), dict(q=both[:9], out=both[:9], lse=both.view(F32).view(-1)[:36].view(9, 4)))
    leaf = torch.zeros((9, 4, 64), dtype=BF16, requires_grad=True)
    with pytest.raises(ValueError, match="requires grad"):
        _prompt(q=leaf)
    with torch.no_grad():
        _prompt(q=leaf)


def _quantize(**kw):
    a = dict(x=torch.zeros((3, 144)))
    a.update(kw)
    return B.mk_quantize_fp8_args.from_buffer_copy(S.native().check_quantize(**a))


def test_quantize_tensors():
    a = _quantize()
    assert (a.m, a.k, a.x_row, a.codes_row, a.scales_row) == (3, 144, 144, 144, 2)
    c = torch.zeros((3, 160)).to(E4M3)[:, :144]
    assert _quantize(codes=c, scales=torch.zeros((3, 5))[:, 1:3]).codes_row == 160
    assert _quantize(x=torch.zeros((1, 144)).expand(3, -1)).x_row == 0
    refused(_quantize, dict(x=torch.zeros((3, 140))), dict(x=torch.zeros((3, 0))), dict(x=torch.zeros((3, 144), dtype=torch.float16)), dict(x=torch.zeros(144)),
            dict(x=torch.zeros((144, 3)).t()), dict(x=torch.zeros((3, 146))[:, :144]), dict(x=torch.zeros(433)[1:].view(3, 144)), dict(codes=torch.zeros((3, 144))),
            dict(codes=torch.zeros((3, 152)).to(E4M3)[:, :144]), dict(codes=torch.zeros((1, 144)).to(E4M3).expand(3, -1)), dict(scales=torch.zeros((3, 1))),
            dict(scales=torch.zeros((2, 3)).t()), dict(scales=torch.zeros((3, 2), dtype=BF16)))
    x = torch.zeros((3, 144))
    refused(_quantize, dict(x=x, scales=x[:, :2]), dict(x=x, codes=x.view(E4M3)[:, :144]))


def _matmul(**kw):
    a = dict(x=torch.zeros((3, 144)).to(E4M3), x_scale=torch.zeros((3, 2)), w=torch.zeros((200, 144)).to(E4M3), w_scale=torch.zeros((2, 2)))
    a.update(kw)
    return B.mk_matmul_fp8_args.from_buffer_copy(S.native().check_matmul(**a))


def test_matmul_tensors():
    a = _matmul()
    assert (a.m, a.n, a.k, a.dtype, a.x_row, a.w_row) == (3, 200, 144, 1, 144, 144)
    assert _matmul(dtype=F32).dtype == 0 and _matmul(out=torch.zeros((3, 200))).dtype == 0 and _matmul(residual=torch.zeros((3, 201))[:, :200]).residual_row == 201
    r = torch.zeros((3, 200), dtype=BF16)
    assert _matmul(residual=r, out=r).y == r.data_ptr()
    wide = torch.zeros((3, 160)).to(E4M3)
    assert _matmul(x=wide[:, :144]).x_row == 160
    refused(_matmul, dict(x=torch.zeros((3, 144))), dict(x=torch.zeros((3, 128)).to(E4M3)), dict(x=torch.zeros((3, 152)).to(E4M3)[:, :144]),
            dict(x=torch.zeros((1, 144)).to(E4M3).expand(3, -1)), dict(w=torch.zeros((1, 144)).to(E4M3).expand(200, -1)), dict(x_scale=torch.zeros((3, 1))),
            dict(x_scale=torch.zeros((3, 2), dtype=BF16)), dict(w_scale=torch.zeros((200, 2))), dict(w_scale=torch.zeros((2, 4))[:, ::2]), dict(w=torch.zeros((200, 144))),
            dict(dtype=torch.float16), dict(dtype=3), dict(dtype=F32, out=torch.zeros((3, 200), dtype=BF16)), dict(residual=torch.zeros((3, 199))),
            dict(out=torch.zeros((3, 200)), residual=torch.zeros((3, 200), dtype=BF16)), dict(out=torch.zeros((200, 3)).t()), dict(out=torch.zeros((1, 200)).expand(3, -1)))
    k = dict(x=torch.zeros((3, 136)).to(E4M3), w=torch.zeros((200, 136)).to(E4M3))
    refused(_matmul, k, dict(x=wide[:, :144], out=wide.view(-1)[:480].view(F32).view(3, 40), w=torch.zeros((40, 144)).to(E4M3), w_scale=torch.zeros((1, 2))))
    buf = torch.zeros(1210)
    refused(_matmul, dict(residual=buf[:600].view(3, 200), out=buf[100:700].view(3, 200)))


def _logits(**kw):
    a = dict(logits=torch.zeros((3, 100)), tokens=i32(3, 20), lengths=i32(3), prompts=i32(3), repetition=torch.ones(3), presence=torch.ones(3),
             frequency=torch.ones(3), bias_ids=i32(3, 4), bias=torch.zeros((3, 4)), mask=i32(3, 4), out=torch.zeros((3, 100)))
    a.update(kw)
    return B.mk_logits_args.from_buffer_copy(S.native().check_logits(**a))


def test_logits_tensors():
    a = _logits()
    assert (a.n, a.vocab, a.columns, a.biases, a.x_row, a.mask_row) == (3, 100, 20, 4, 100, 4)
    assert _logits(mask=i32(1, 4).expand(3, -1)).mask_row == 0
    x = torch.zeros((3, 101), dtype=BF16)[:, 1:]
    assert _logits(logits=x, out=x).x_row == 101
    off = dict(tokens=None, prompts=None, repetition=None, presence=None, frequency=None)
    assert _logits(**off).columns == 0
    refused(_logits, dict(logits=torch.zeros((3, 100), dtype=torch.float16)), dict(logits=torch.zeros(100)), dict(logits=torch.zeros((100, 3)).t()),
            dict(tokens=i32(2, 20)), dict(tokens=i32(3, 20).long()), dict(tokens=i32(20, 3).t()), dict(tokens=None), dict(off, prompts=i32(3)),
            dict(off, presence=torch.ones(3)), dict(lengths=i32(4)), dict(repetition=torch.ones(2)), dict(frequency=torch.ones(3, dtype=BF16)), dict(bias=None),
            dict(bias_ids=None), dict(bias=torch.zeros((3, 5))), dict(mask=i32(3, 3)), dict(mask=i32(3, 4).bool()), dict(out=torch.zeros((3, 99))),
            dict(out=torch.zeros((3, 100), dtype=BF16)), dict(out=torch.zeros((1, 100)).expand(3, -1)))
    buf = torch.zeros(700)
    refused(_logits, dict(logits=buf[:300].view(3, 100), out=buf[1:301].view(3, 100)), dict(out=buf[:300].view(3, 100), repetition=buf[10:13]),
            dict(out=buf[:300].view(3, 100), mask=buf.view(torch.int32)[290:302].view(3, 4)))


def test_sinks_of_single_tokens():
    f = lambda **kw: B.mk_attention_args.from_buffer_copy(S.native().check_attention(**dict(CACHE, q=torch.zeros((3, 4, 64)), lengths=i32(3), **kw)))  # noqa: E731
    assert f().sinks == 0 and f(window=9, sinks=4).sinks == 4 and f(window=9, sinks=2 ** 40).sinks == 2 ** 31 - 1
    refused(f, dict(sinks=-1), dict(window=3, sinks=-5))


def test_the_functions_describe_themselves():
    for n in S.NATIVE:
        f = getattr(mk, n)
        assert "stream" in inspect.signature(f).parameters and f.__name__ in f.__doc__
    assert "sinks" in inspect.signature(mk.paged_attention).parameters


def test_argument_errors_of_the_c_entry_points():
    # returned before any CUDA call; the pointers are never followed
    lib = mk.load_library()

    def with_(s, f):
        for k, v in f.items():
            setattr(s, k, v)
        return C.byref(s)

    def plan(**f):
        a = B.mk_plan_args(n=2, rows=5, page_size=16, lengths=16, counts=16, table=16, table_cols=4, table_stride=4, free=16, free_count=3, used=16, seqs=16,
                           slots=16, starts=16, totals=16, used_out=16)
        return lib.mk_paged_plan(with_(a, f), None)
    assert lib.mk_paged_plan(None, None) == -1
    for f in (dict(n=-1), dict(rows=-1), dict(page_size=0), dict(lengths=None), dict(table=None), dict(table_cols=-1), dict(table_stride=-1), dict(free=None),
              dict(free_count=-1), dict(used=None), dict(seqs=None), dict(slots=None), dict(starts=None), dict(totals=None), dict(used_out=None), dict(counts=None)):
        assert plan(**f) == -1, f
    assert plan(n=16385) == -2

    kv = B.mk_paged_kv(16, 16, 1, 4, 2, 16, 64, 2048, 1024, 64, None, None, 16, 3, 4, 4)

    def prompt(kv=kv, **f):
        a = B.mk_prompt_args(n=2, rows=0, dtype=1, n_q_heads=4, q=16, out=16, q_row=256, q_head=64, out_row=256, out_head=64, starts=16, lengths=16, scale=0.125)
        return lib.mk_paged_prompt_attention(C.byref(kv), with_(a, f), None)
    assert prompt() == 0 and prompt(rows=4, n=0) == 0
    assert lib.mk_paged_prompt_attention(None, None, None) == -1 and lib.mk_paged_prompt_attention(C.byref(kv), None, None) == -1
    for f in (dict(n=-1), dict(n=4), dict(rows=-1), dict(dtype=2), dict(n_q_heads=3), dict(n_q_heads=0), dict(window=-1), dict(sinks=-1), dict(scale=float("inf")),
              dict(rows=1, q=None), dict(rows=1, out=24), dict(rows=1, starts=None), dict(rows=1, lengths=None), dict(rows=1, q_row=12), dict(rows=1, out_head=-8)):
        assert prompt(**f) == -1, f
    assert prompt(dtype=0) == -2 and prompt(rows=2 ** 31 - 1) == -2
    assert prompt(B.mk_paged_kv(16, 16, 1, 4, 2, 16, 96, 2048, 1024, 64, None, None, 16, 3, 4, 4)) == -2
    assert prompt(B.mk_paged_kv(16, 16, 1, 4, 2, 16, 64, 2048, 1024, 64, None, None, 16, 3, 2 ** 28, 4), rows=1) == -2
    assert lib.mk_paged_prompt_attention_workspace(2, 9, 4, 2, 96) == -2 and lib.mk_paged_prompt_attention_workspace(2, 9, 3, 2, 64) == -1
    asked = []
    ask = B.WORKSPACE_FN(lambda context, n: asked.append(n))
    empty = B.mk_prompt_args(n=2, rows=0, dtype=1, n_q_heads=4, q=16, out=16, starts=16, lengths=16, scale=0.125)
    assert lib.mk_paged_prompt_attention_ask(C.byref(kv), C.byref(empty), ask, None, None) == 0 and not asked
    assert lib.mk_paged_prompt_attention_ask(C.byref(kv), C.byref(empty), B.WORKSPACE_FN(0), None, None) == -1

    def quantize(**f):
        return lib.mk_quantize_fp8(with_(B.mk_quantize_fp8_args(m=0, k=144, dtype=0, x=16, x_row=144, codes=16, codes_row=144, scales=16, scales_row=2), f), None)
    assert quantize() == 0 and lib.mk_quantize_fp8(None, None) == -1
    for f in (dict(m=-1), dict(k=0), dict(k=24), dict(dtype=2), dict(m=1, x=None), dict(m=1, x=24), dict(m=1, codes=8), dict(m=1, scales=None), dict(m=1, x_row=146),
              dict(m=1, codes_row=152), dict(x_row=-16), dict(scales_row=-1)):
        assert quantize(**f) == -1, f

    def matmul(**f):
        a = B.mk_matmul_fp8_args(m=0, n=8, k=144, dtype=0, x=16, x_row=144, x_scale=16, x_scale_row=2, w=16, w_row=144, w_scale=16, y=16, y_row=8)
        return lib.mk_matmul_fp8(with_(a, f), None)
    assert matmul() == 0 and matmul(m=1, n=0) == 0 and lib.mk_matmul_fp8(None, None) == -1
    for f in (dict(m=-1), dict(n=-1), dict(k=0), dict(k=24), dict(dtype=2), dict(m=1, x=None), dict(m=1, x=24), dict(m=1, w=8), dict(m=1, x_scale=None),
              dict(m=1, w_scale=None), dict(m=1, y=None), dict(m=1, y=2), dict(m=1, residual=2), dict(m=1, x_row=128), dict(m=1, w_row=152), dict(y_row=-1)):
        assert matmul(**f) == -1, f

    def logits(**f):
        return lib.mk_adjust_logits(with_(B.mk_logits_args(n=0, vocab=8, dtype=0, x=16, out=16, x_row=8, out_row=8), f), None)
    assert logits() == 0 and logits(n=1, vocab=0) == 0 and lib.mk_adjust_logits(None, None) == -1
    for f in (dict(n=-1), dict(vocab=-1), dict(dtype=2), dict(columns=-1), dict(biases=-1), dict(n=1, x=None), dict(n=1, out=18), dict(n=1, columns=3),
              dict(n=1, biases=2), dict(n=1, biases=2, bias_ids=16), dict(mask_row=-1), dict(x_row=-8)):
        assert logits(**f) == -1, f


def test_quantised_weights():
    w = torch.randn((200, 272), generator=torch.Generator().manual_seed(0)) * 0.02
    w[128:, 128:256] = 0.0
    codes, scales = mk.quantize_fp8_weight(w)
    assert codes.shape == w.shape and codes.dtype == E4M3 and scales.shape == (2, 3) and scales[1, 1] == 1
    for a in range(2):
        for b in range(3):
            part = w[a * 128:(a + 1) * 128, b * 128:(b + 1) * 128].double()
            s = (part.abs().max() / 448).float().double()
            if s == 0:
                continue
            assert scales[a, b].double() == s
            # half a step of e4m3: 2^-4 of the value, 2^-10 below its normal numbers
            off = (codes[a * 128:(a + 1) * 128, b * 128:(b + 1) * 128].double() * s - part).abs()
            assert (off <= torch.maximum(part.abs() * 2.0 ** -4, s * 2.0 ** -10) * (1 + 2.0 ** -20)).all()
    with pytest.raises(ValueError):
        mk.quantize_fp8_weight(w[:, :200])


def test_the_plain_forms_agree_with_themselves():
    # the bisected plan of a small step by hand; a mistake planted in the plain form shows
    got = P.plan([3, -1, 4, 0], [2, 5, 1, 0], [[9, -1], [-1, -1], [8, -1], [-1, -1]], [5, 6, 7], 1, 4, 6)
    assert got == ([0, 0, 2, -1, -1, -1], [3, 4, 4, -1, -1, -1], [0, 2, 2, 3, 3], [5, -1, 5, 0], 3, [[9, 6], [-1, -1], [8, 7], [-1, -1]], True)
    assert P.plan([3], [2], [[9, -1]], [5, 6], 2, 4, 6)[-1] is False
    x = torch.randn((3, 40))
    codes, s = P.quantized(x)
    assert (codes == (x / s.float()).to(E4M3).double()).all()
    assert not (codes == (x / (s.float() * 1.1)).to(E4M3).double()).all()
