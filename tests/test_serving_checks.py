"""Refusals of the paged-cache and 4-bit operators, and their host logic (no GPU)."""
import ctypes as C
import os

import pytest
import torch

import serving_util as U

import persistent_transformer_megakernel_gb300 as mk
from persistent_transformer_megakernel_gb300 import _binding as B
from persistent_transformer_megakernel_gb300 import serving as S

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


if not os.path.exists(mk.lib_path()) or not os.path.exists(os.path.join(os.path.dirname(mk.lib_path()), "_mktorch.so")):
    from persistent_transformer_megakernel_gb300 import build
    build.build()

CACHE = dict(k_cache=torch.zeros((6, 2, 16, 64), dtype=BF16), v_cache=torch.zeros((6, 2, 16, 64), dtype=BF16),
             table=torch.zeros((3, 4), dtype=torch.int32))


def _kv(**kw):
    a = dict(k_cache=torch.zeros((6, 2, 16, 64), dtype=BF16), v_cache=torch.zeros((6, 2, 16, 64), dtype=BF16),
             table=torch.zeros((3, 4), dtype=torch.int32))
    a.update(kw)
    return S.paged_struct(**a, on_device=False)


def test_cache_tensors():
    kv = _kv()
    assert (kv.n_pages, kv.n_kv_heads, kv.page_size, kv.head_dim) == (6, 2, 16, 64)
    assert (kv.page_stride, kv.head_stride, kv.slot_stride, kv.table_stride) == (2048, 1024, 64, 4)
    t = lambda *s, dtype=BF16: torch.zeros(s, dtype=dtype)  # noqa: E731
    both = t(6, 2, 16, 2, 64)                                   # keys and values of a page together, slots before heads
    assert _kv(k_cache=both[:, 0].transpose(1, 2), v_cache=both[:, 1].transpose(1, 2)).slot_stride == 128
    assert _kv(table=torch.zeros((1, 4), dtype=torch.int32).expand(3, -1)).table_stride == 0
    f8 = t(6, 2, 16, 64, dtype=E4M3)
    one = torch.ones(2)
    assert _kv(k_cache=f8, v_cache=f8, k_scale=one, v_scale=one).dtype == 2
    for bad in (dict(k_cache=t(6, 2, 16, 64, dtype=F32)), dict(v_cache=t(6, 2, 16, 64, dtype=E4M3)), dict(v_cache=t(5, 2, 16, 64)),
                dict(k_cache=t(6, 2, 16, 96), v_cache=t(6, 2, 16, 96)), dict(k_cache=t(2, 16, 64), v_cache=t(2, 16, 64)),
                dict(k_cache=t(6, 2, 64, 16).transpose(2, 3), v_cache=t(6, 2, 64, 16).transpose(2, 3)),
                dict(k_cache=t(6, 2, 16, 68)[..., :64], v_cache=t(6, 2, 16, 68)[..., :64]),
                dict(k_cache=t(12288 + 4)[4:].view(6, 2, 16, 64)), dict(k_cache=t(0, 2, 16, 64), v_cache=t(0, 2, 16, 64)),
                dict(table=torch.zeros((3, 4), dtype=torch.int64)), dict(table=torch.zeros(4, dtype=torch.int32)),
                dict(table=torch.zeros((4, 3), dtype=torch.int32).t()), dict(k_scale=one), dict(k_scale=one, v_scale=one),
                dict(k_cache=f8, v_cache=f8, k_scale=one), dict(k_cache=f8, v_cache=f8, k_scale=one, v_scale=torch.ones(3)),
                dict(k_cache=f8, v_cache=f8, k_scale=one, v_scale=one.double())):
        with pytest.raises(ValueError):
            _kv(**bad)
    with pytest.raises(ValueError):                             # host tensors
        S.paged_struct(t(6, 2, 16, 64), t(6, 2, 16, 64), torch.zeros((3, 4), dtype=torch.int32))


def _append(**kw):
    a = dict(CACHE, k=torch.zeros((3, 2, 64)), v=torch.zeros((3, 2, 64)), slots=torch.zeros(3, dtype=torch.int32), seqs=None,
             q=torch.zeros((3, 4, 64)), q_out=torch.zeros((3, 4, 64)), rope=torch.zeros((10, 32, 2)), positions=None,
             mrope_sections=None, mrope_interleaved=False, q_norm=torch.zeros(64, dtype=BF16), k_norm=None, eps=1e-6, status=None)
    a.update(kw)
    return B.mk_append_args.from_buffer_copy(S.native().check_append(**a))


def test_append_tensors():
    a = _append()
    assert (a.n, a.n_q_heads, a.rope_rows, a.rope_mode, a.k_row) == (3, 4, 10, 0, 128)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    assert _append(positions=i32(3, 3), mrope_sections=(12, 10, 10), mrope_interleaved=True).rope_mode == 2
    assert _append(q=None, q_out=None, rope=None).n_q_heads == 0
    stacked = torch.zeros((3, 8, 64))
    assert _append(q=stacked[:, :4], k=stacked[:, 4:6], v=stacked[:, 6:]).k_row == 512
    assert _append(seqs=i32(3)).seqs
    four = dict(k=torch.zeros((4, 2, 64)), v=torch.zeros((4, 2, 64)), slots=i32(4), q=None, q_out=None)
    with pytest.raises(ValueError):                             # row 3 has no table row
        _append(**four)
    assert _append(**four, seqs=i32(4)).n == 4
    for bad in (dict(k=torch.zeros((3, 2, 64), dtype=torch.float16)), dict(v=torch.zeros((3, 2, 64), dtype=BF16)),
                dict(k=torch.zeros((3, 3, 64)), v=torch.zeros((3, 3, 64))), dict(v=torch.zeros((2, 2, 64))),
                dict(k=torch.zeros((3, 2, 66))[..., :64]), dict(k=torch.zeros((3, 64, 2)).transpose(1, 2)),
                dict(k=torch.zeros(3 * 128 + 1)[1:].view(3, 2, 64)), dict(q_out=torch.zeros((3, 3, 64))),
                dict(q_out=torch.zeros((3, 4, 64), dtype=BF16)), dict(q=torch.zeros((3, 256))), dict(slots=i32(2)), dict(slots=None),
                dict(slots=torch.zeros(3, dtype=torch.int64)), dict(seqs=i32(2)), dict(rope=torch.zeros((10, 32))),
                dict(rope=torch.zeros((10, 64, 2))), dict(rope=torch.zeros((10, 32, 2), dtype=torch.float64)), dict(positions=i32(2)),
                dict(positions=i32(3, 3)), dict(mrope_sections=(12, 10, 10)), dict(positions=i32(3, 3), mrope_sections=(12, 10, 9)),
                dict(positions=i32(3, 3), mrope_sections=(42, -5, -5)), dict(positions=i32(3, 4), mrope_sections=(12, 10, 10)),
                dict(rope=None, positions=i32(3)), dict(q_norm=torch.zeros(64)), dict(k_norm=torch.zeros(128, dtype=BF16)), dict(k_norm=torch.zeros(65, dtype=BF16)[1:]),
                dict(status=i32(2)), dict(q=None), dict(eps=-1.0), dict(eps=float("nan")), dict(v=None), dict(mrope_sections=(16, 16))):
        with pytest.raises(ValueError):
            _append(**bad)
    for bad in (dict(eps="x"), dict(positions=i32(3, 3), mrope_sections=3), dict(nonsense=1)):
        with pytest.raises(TypeError):
            _append(**bad)
    with pytest.raises(TypeError):
        mk.paged_append(stacked)
    with pytest.raises(ValueError):                             # host tensors where device ones are needed
        mk.paged_append(stacked[:, 4:6], stacked[:, 6:], *CACHE.values(), i32(3))


def _attention(**kw):
    a = dict(CACHE, q=torch.zeros((3, 4, 64)), lengths=torch.zeros(3, dtype=torch.int32), scale=None, window=0,
             out=torch.zeros((3, 4, 64)), lse=torch.zeros((3, 4)), status=None)
    a.update(kw)
    return B.mk_attention_args.from_buffer_copy(S.native().check_attention(**a))


def test_attention_tensors():
    a = _attention()
    assert (a.n, a.n_q_heads, a.scale) == (3, 4, 0.125)
    assert _attention(q=torch.zeros((3, 8, 64))[:, ::2]).q_head == 128
    for bad in (dict(q=torch.zeros((3, 3, 64))), dict(q=torch.zeros((3, 4, 128))), dict(q=torch.zeros((3, 0, 64))),
                dict(q=torch.zeros((4, 4, 64)), out=torch.zeros((4, 4, 64)), lse=None, lengths=torch.zeros(4, dtype=torch.int32)),
                dict(q=torch.zeros((3, 4, 64), dtype=torch.float16)), dict(out=torch.zeros((3, 4, 64), dtype=BF16)),
                dict(out=torch.zeros((3, 2, 64))), dict(lse=torch.zeros((4, 3)).t()), dict(lse=torch.zeros((3, 4), dtype=BF16)),
                dict(lengths=torch.zeros(3)), dict(lengths=torch.zeros(4, dtype=torch.int32)), dict(lengths=None), dict(window=-1),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None), dict(q=3)):
        with pytest.raises(ValueError):
            _attention(**bad)


def _matvec(**kw):
    a = dict(x=torch.zeros((2, 128)), codes=torch.zeros((10, 64), dtype=torch.uint8), scales=torch.zeros((10, 2), dtype=BF16),
             zeros=None, residual=None, out=torch.zeros((2, 10)))
    a.update(kw)
    return B.mk_matvec_q4_args.from_buffer_copy(S.native().check_matvec(**a))


def test_matvec_tensors():
    a = _matvec()
    assert (a.m, a.n, a.k, a.group) == (2, 10, 128, 64)
    assert _matvec(scales=torch.zeros((10, 4), dtype=BF16), zeros=torch.zeros((10, 4), dtype=torch.uint8)).group == 32
    assert _matvec(residual=torch.zeros((2, 11))[:, :10]).residual_row == 11
    assert _matvec(x=torch.zeros((1, 128)).expand(2, -1)).x_row == 0
    for bad in (dict(x=torch.zeros((2, 64))), dict(x=torch.zeros((2, 128), dtype=torch.float16)), dict(x=torch.zeros((128, 2)).t()),
                dict(x=torch.zeros((2, 130))[:, :128]), dict(x=torch.zeros(257)[1:].view(2, 128)),
                dict(codes=torch.zeros((10, 64), dtype=torch.int8)), dict(codes=torch.zeros((64, 10), dtype=torch.uint8).t()),
                dict(scales=torch.zeros((10, 2))), dict(scales=torch.zeros((9, 2), dtype=BF16)), dict(scales=torch.zeros((10, 8), dtype=BF16)),
                dict(scales=torch.zeros((10, 3), dtype=BF16)), dict(zeros=torch.zeros((10, 1), dtype=torch.uint8)),
                dict(zeros=torch.zeros((10, 2))), dict(residual=torch.zeros((2, 9))), dict(residual=torch.zeros((2, 10), dtype=BF16)),
                dict(out=torch.zeros((3, 10))), dict(out=torch.zeros((2, 10), dtype=BF16)), dict(out=torch.zeros((10, 2)).t())):
        with pytest.raises(ValueError):
            _matvec(**bad)
    with pytest.raises(ValueError):                             # host tensors
        mk.matvec_q4(torch.zeros((2, 128)), torch.zeros((10, 64), dtype=torch.uint8), torch.zeros((10, 2), dtype=BF16))


def test_the_functions_describe_themselves():
    import inspect
    for f in (mk.paged_append, mk.paged_attention, mk.matvec_q4):
        assert "stream" in inspect.signature(f).parameters and f.__name__ in f.__doc__
    with pytest.raises(AttributeError):
        mk.no_such_operator


def _with(s, fields):
    for k, v in fields.items():
        setattr(s, k, v)
    return s


def test_argument_errors_of_the_c_entry_points():
    # returned before any CUDA call; the pointers are never followed
    if not os.path.exists(mk.lib_path()):
        pytest.skip("library not built")
    lib = mk.load_library()
    assert lib.mk_error_string(-10).startswith(b"page")

    def kv(**f):
        return _with(B.mk_paged_kv(16, 16, 1, 4, 2, 16, 64, 2048, 1024, 64, None, None, 16, 3, 4, 4), f)

    def app(**f):
        return _with(B.mk_append_args(n=0, dtype=0, k=16, v=16, slots=16, k_row=128, k_head=64, v_row=128, v_head=64), f)

    def att(**f):
        return _with(B.mk_attention_args(n=0, dtype=0, n_q_heads=4, q=16, out=16, q_row=256, q_head=64, out_row=256, out_head=64,
                                         lengths=16, scale=0.125, workspace=16, workspace_bytes=0), f)

    def append(k, a):
        return lib.mk_paged_append(C.byref(k), C.byref(a), None)

    def attend(k, a):
        return lib.mk_paged_attention(C.byref(k), C.byref(a), None)

    assert append(kv(), app()) == 0 and attend(kv(), att()) == 0       # no rows: nothing to do
    assert lib.mk_paged_append(None, None, None) == -1 and lib.mk_paged_attention(None, None, None) == -1
    assert lib.mk_paged_append(C.byref(kv()), None, None) == -1
    for f in (dict(k=None), dict(v=24), dict(dtype=0), dict(n_pages=0), dict(n_kv_heads=0), dict(page_size=0), dict(page_stride=-8),
              dict(slot_stride=7), dict(table=None), dict(table_rows=-1), dict(k_scale=16), dict(k_scale=16, v_scale=16), dict(table_stride=-1)):
        assert append(kv(**f), app()) == -1 and attend(kv(**f), att()) == -1, f
    assert append(kv(head_dim=96), app()) == -2 and attend(kv(head_dim=96), att()) == -2
    for f in (dict(n=-1), dict(dtype=2), dict(n=1, k=None), dict(n=1, v=8), dict(n=1, slots=None), dict(n=1, k_row=130), dict(n=1, v_head=-4),
              dict(n=1, n_q_heads=2), dict(rope_mode=3), dict(rope_rows=-1), dict(n=1, rope=16, rope_rows=4, rope_mode=1),
              dict(n=1, k_norm=16, rms_eps=-1.0), dict(n=1, q_norm=18, rms_eps=0.0), dict(n=1, rope=8, rope_rows=4)):
        assert append(kv(), app(**f)) == -1, f
    for f in (dict(n=4), dict(n=-1), dict(dtype=2), dict(window=-1), dict(n_q_heads=3), dict(n_q_heads=0), dict(scale=float("nan")),
              dict(scale=float("inf")), dict(n=1, q=None), dict(n=1, out=20), dict(n=1, lengths=None), dict(n=1, workspace=None),
              dict(n=1, out_row=6)):
        assert attend(kv(), att(**f)) == -1, f
    assert attend(kv(table_cols=2 ** 30), att(n=1)) == -2               # more slots than a length can say
    assert lib.mk_paged_attention_workspace(4, 3, 64) == -1 and lib.mk_paged_attention_workspace(4, 2, 80) == -2

    def mv(**f):
        return lib.mk_matvec_q4(C.byref(_with(B.mk_matvec_q4_args(0, 8, 128, 64, 0, 16, 128, 16, 16, None, None, 0, 16, 8), f)), None)

    assert mv() == 0 and mv(m=1, n=0) == 0 and lib.mk_matvec_q4(None, None) == -1
    for f in (dict(m=-1), dict(n=-1), dict(k=0), dict(group=0), dict(group=96), dict(dtype=2), dict(m=1, x=None), dict(m=1, x=8),
              dict(m=1, codes=24), dict(m=1, scales=None), dict(m=1, y=None), dict(m=1, x_row=130), dict(m=1, y_row=-1)):
        assert mv(**f) == -1, f
    assert mv(group=16) == -2 and mv(group=128, k=32896) == -2 and mv(k=192, group=192) == -2
    assert lib.mk_export_kv(None, 0, 0, 0, None, 0, 0, None) == -1


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_quantised_weights(group, zeros):
    w = torch.randn((6, 256), generator=torch.Generator().manual_seed(0)) * 0.02 + (0.02 if zeros else 0.0)
    w[2] = 0.0
    q = mk.quantize_q4(w, group, zeros)
    back = U.dequantize(*q)
    s = q[1].double().repeat_interleave(group, 1)
    # nearest code: half a scale; the scale's rounding to bf16 (2^-8 of 7, or of 15, codes) and the zero's to a whole
    # number can push the ends of a group past the last code
    assert ((back - w.double()).abs() <= s * (0.5 + (15 * 2.0 ** -8 + 1.0 if zeros else 7 * 2.0 ** -8)) + 1e-12).all()
    assert (back[2] == 0).all()
    with pytest.raises(ValueError):
        mk.quantize_q4(w, 48)
    with pytest.raises(ValueError):
        mk.quantize_q4(w[:, :200], 64)


def test_rope_table():
    t = mk.rope_table(5, 64, device="cpu")
    a = U.rotary(torch.arange(5), 64)
    assert t.shape == (5, 32, 2) and t.dtype == F32
    assert torch.equal(t[..., 0], a.cos().float()) and torch.equal(t[..., 1], a.sin().float())


def test_what_is_written_is_not_expanded():
    for kw in (dict(q_out=torch.zeros((1, 4, 64)).expand(3, -1, -1)), dict(q_out=torch.zeros((3, 1, 64)).expand(-1, 4, -1)),
               dict(k_cache=torch.zeros((1, 2, 16, 64), dtype=BF16).expand(6, -1, -1, -1), v_cache=torch.zeros((1, 2, 16, 64), dtype=BF16).expand(6, -1, -1, -1))):
        with pytest.raises(ValueError, match="expanded"):
            _append(**kw)
    for out in (torch.zeros((1, 4, 64)).expand(3, -1, -1), torch.zeros((3, 1, 64)).expand(-1, 4, -1)):
        with pytest.raises(ValueError, match="expanded"):
            _attention(q=torch.zeros((3, 4, 64)), out=out)
    x = torch.zeros((3, 128))
    codes, scales = torch.zeros((128, 64), dtype=torch.uint8), torch.zeros((128, 2), dtype=BF16)
    with pytest.raises(ValueError, match="expanded"):
        _matvec(x=x, codes=codes, scales=scales, residual=None, zeros=None, out=torch.zeros((1, 128)).expand(3, -1))
    with pytest.raises(ValueError, match="must not be x"):
        _matvec(x=x, codes=codes, scales=scales, residual=None, zeros=None, out=x)
    _matvec(x=x, codes=codes, scales=scales, residual=x, zeros=None, out=torch.zeros((3, 128)))


def test_a_call_that_asks_for_its_workspace_checks_the_same():
    lib = B.load_library()
    asked = []
    ask = B.WORKSPACE_FN(lambda context, n: asked.append(n))
    kv = B.mk_paged_kv.from_buffer_copy(bytes(_kv()))
    a = _attention(lse=None)
    for field, value in (("n", 4), ("q", None), ("lengths", None), ("dtype", 7), ("scale", float("inf")), ("n_q_heads", 3)):
        b = B.mk_attention_args.from_buffer_copy(bytes(a))
        setattr(b, field, value)
        assert lib.mk_paged_attention_ask(C.byref(kv), C.byref(b), ask, None, None) == -1
    assert lib.mk_paged_attention_ask(C.byref(kv), C.byref(a), B.WORKSPACE_FN(0), None, None) == -1
    assert lib.mk_paged_attention_ask(None, C.byref(a), ask, None, None) == -1
    a.n = 0
    assert lib.mk_paged_attention_ask(C.byref(kv), C.byref(a), ask, None, None) == 0 and not asked
