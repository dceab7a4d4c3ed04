"""Calls of the batched serving operators that are refused because their results
would not be what the call says (no GPU: the checks alone)."""
import os

import pytest
import torch

import persistent_transformer_megakernel_gb300 as mk
from persistent_transformer_megakernel_gb300 import _binding as B
from persistent_transformer_megakernel_gb300 import serving as S

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn

if not os.path.exists(mk.lib_path()) or not os.path.exists(os.path.join(os.path.dirname(mk.lib_path()), "_mktorch.so")):
    from persistent_transformer_megakernel_gb300 import build
    build.build()


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _cache(**kw):
    return dict(dict(k_cache=torch.zeros((6, 2, 16, 64), dtype=BF16), v_cache=torch.zeros((6, 2, 16, 64), dtype=BF16), table=_i32(3, 4)), **kw)


def _append(**kw):
    a = dict(_cache(), k=torch.zeros((3, 2, 64)), v=torch.zeros((3, 2, 64)), slots=_i32(3), q=torch.zeros((3, 4, 64)))
    a.update(kw)
    return B.mk_append_args.from_buffer_copy(S.native().check_append(**a))


def _attention(**kw):
    a = dict(_cache(), q=torch.zeros((3, 4, 64)), lengths=_i32(3))
    a.update(kw)
    return B.mk_attention_args.from_buffer_copy(S.native().check_attention(**a))


def _matvec(**kw):
    a = dict(x=torch.zeros((3, 128)), codes=torch.zeros((10, 64), dtype=torch.uint8), scales=torch.zeros((10, 2), dtype=BF16))
    a.update(kw)
    return B.mk_matvec_q4_args.from_buffer_copy(S.native().check_matvec(**a))


def test_a_rotary_table_without_rows():
    assert _append(rope=torch.zeros((1, 32, 2))).rope
    for kw in (dict(), dict(positions=_i32(3)), dict(positions=_i32(3, 3), mrope_sections=(12, 10, 10))):
        with pytest.raises(ValueError, match="rope"):
            _append(rope=torch.zeros((0, 32, 2)), **kw)


def test_queries_are_written_in_place_or_apart():
    buf = torch.zeros(4000)
    q = buf[:768].view(3, 4, 64)
    for make in (lambda out: _append(q=q, q_out=out), lambda out: _attention(q=q, out=out)):
        make(q)                                             # itself
        make(buf[768:1536].view(3, 4, 64))                  # behind it
        for out in (buf[64:832].view(3, 4, 64), buf[4:772].view(3, 4, 64),
                    torch.as_strided(buf, (3, 4, 64), (320, 64, 1)), torch.as_strided(buf, (3, 4, 64), (64, 192, 1)),
                    torch.as_strided(buf, (3, 4, 64), (256, 64, 1), 512)):
            with pytest.raises(ValueError, match="overlap"):
                make(out)
    # pieces of the same rows: beside one another, heads between heads, the halves of a buffer of heads
    wide = torch.zeros((3, 8, 64))
    for a, b in ((wide[:, :4], wide[:, 4:]), (wide[:, ::2], wide[:, 1::2])):
        for x, y in ((a, b), (b, a)):
            _append(q=x, q_out=y)
            _attention(q=x, out=y)
    two = torch.zeros((3, 4, 128))
    _attention(q=two[..., :64], out=two[..., 64:])
    by_head = torch.zeros((8, 3, 64)).transpose(0, 1)
    _attention(q=by_head[:, :4], out=by_head[:, 4:])
    with pytest.raises(ValueError, match="overlap"):
        _attention(q=wide[:, :4], out=wide[:, 2:6])


def test_queries_are_not_written_over_keys_values_or_the_cache():
    qkv = torch.zeros((3, 8, 64))
    a = dict(q=qkv[:, :4], k=qkv[:, 4:6], v=qkv[:, 6:])
    _append(**a, q_out=qkv[:, :4])
    for out in (qkv[:, 2:6], qkv[:, 4:]):
        with pytest.raises(ValueError, match="overlap"):
            _append(**a, q_out=out)
    cache = torch.zeros((6, 2, 16, 64), dtype=BF16)
    b = dict(k_cache=torch.zeros_like(cache), v_cache=cache, q=torch.zeros((3, 4, 64), dtype=BF16))
    out = cache[1, 0, :12].view(3, 4, 64)
    with pytest.raises(ValueError, match="overlap"):
        _attention(**b, out=out)
    with pytest.raises(ValueError, match="overlap"):
        _append(**b, k=torch.zeros((3, 2, 64), dtype=BF16), v=torch.zeros((3, 2, 64), dtype=BF16), q_out=out)


def test_caches_that_are_written_are_two():
    one = torch.zeros((6, 2, 16, 64), dtype=BF16)
    both = torch.zeros((6, 2, 16, 2, 64), dtype=BF16)
    _append(k_cache=both[:, 0].transpose(1, 2), v_cache=both[:, 1].transpose(1, 2))
    slots = torch.zeros((6, 2, 16, 128), dtype=BF16)
    _append(k_cache=slots[..., :64], v_cache=slots[..., 64:])
    pair = torch.zeros((2, 6, 2, 16, 64), dtype=BF16)
    _append(k_cache=pair[0], v_cache=pair[1])
    _attention(k_cache=one, v_cache=one)                    # only read: keys may be the values
    flat = torch.zeros(20000, dtype=BF16)
    for k, v in ((one, one), (flat[:12288].view(6, 2, 16, 64), flat[2048:14336].view(6, 2, 16, 64)),
                 (torch.as_strided(flat, (6, 2, 16, 64), (2048, 1024, 32, 1)), torch.zeros(20000, dtype=BF16).as_strided((6, 2, 16, 64), (2048, 1024, 32, 1))),
                 (torch.as_strided(flat, (6, 2, 16, 64), (1024, 1024, 64, 1)), torch.zeros(20000, dtype=BF16).as_strided((6, 2, 16, 64), (1024, 1024, 64, 1)))):
        with pytest.raises(ValueError, match="overlap"):
            _append(k_cache=k, v_cache=v)


def test_outputs_that_overlap_themselves():
    flat = torch.zeros(4000)
    for strides in ((256, 32, 1), (128, 64, 1), (64, 64, 1), (60, 256, 1)):
        for make in (lambda out: _append(q_out=out), lambda out: _attention(out=out)):
            with pytest.raises(ValueError, match="overlap|16 bytes"):
                make(torch.as_strided(flat, (3, 4, 64), strides))
    _attention(out=torch.as_strided(flat, (3, 4, 64), (64, 192, 1)))
    with pytest.raises(ValueError, match="overlap"):
        _matvec(out=torch.as_strided(flat, (3, 10), (9, 1)))
    _matvec(out=torch.as_strided(flat, (3, 10), (10, 1)))


def test_the_sums_log_is_apart():
    buf = torch.zeros(2000)
    q = buf[:768].view(3, 4, 64)
    _attention(q=q, lse=buf[768:780].view(3, 4))
    with pytest.raises(ValueError, match="lse"):
        _attention(q=q, lse=buf[760:772].view(3, 4))
    with pytest.raises(ValueError, match="lse"):
        _attention(out=q, lse=buf[:12].view(3, 4))


def test_products_are_written_apart_from_x_and_in_place_of_the_residual():
    buf = torch.zeros((3, 512))
    x = buf[:, :128]
    square = dict(codes=torch.zeros((128, 64), dtype=torch.uint8), scales=torch.zeros((128, 2), dtype=BF16))
    _matvec(x=x, **square, out=buf[:, 128:256])
    for out in (buf[:, 4:132], buf[:, 127:255], x, torch.as_strided(buf, (3, 128), (500, 1), 300), buf.view(-1)[60:444].view(3, 128)):
        with pytest.raises(ValueError, match="must not be x"):
            _matvec(x=x, **square, out=out)
    r = buf[:, 200:328]
    _matvec(x=x, **square, residual=r, out=r)
    _matvec(x=x, **square, residual=r, out=buf[:, 384:])
    for out in (buf[:, 201:329], buf[:, 328 - 1:328 + 127], torch.as_strided(buf, (3, 128), (513, 1), 200)):
        with pytest.raises(ValueError, match="overlap"):
            _matvec(x=x, **square, residual=r, out=out)


def test_strides_of_single_rows_and_heads_do_not_matter():
    # a dimension of one element has a stride that is never used
    odd = torch.zeros(2000)
    row = torch.as_strided(odd, (1, 4, 64), (257, 64, 1))
    a = _append(k=torch.as_strided(odd, (1, 2, 64), (131, 64, 1)), v=torch.as_strided(odd, (1, 2, 64), (7, 64, 1)), slots=_i32(1), q=row,
                q_out=torch.as_strided(torch.zeros(2000), (1, 4, 64), (3, 64, 1)))
    assert a.n == 1 and a.k_row % 4 == a.v_row % 4 == a.q_row % 4 == a.out_row % 4 == 0
    a = _attention(q=row, lengths=_i32(1), out=row)
    assert a.q_row == a.out_row
    head = torch.as_strided(odd, (3, 1, 64), (64, 1, 1))
    one = dict(k_cache=torch.zeros((6, 1, 16, 64), dtype=BF16), v_cache=torch.zeros((6, 1, 16, 64), dtype=BF16))
    assert _attention(**one, q=head, out=torch.as_strided(torch.zeros(300), (3, 1, 64), (64, 5, 1))).q_head % 4 == 0
    # in place by another view of the same memory
    _attention(q=row, lengths=_i32(1), out=torch.as_strided(odd, (1, 4, 64), (256, 64, 1)))
    a = _matvec(x=torch.as_strided(odd, (1, 128), (129, 1)), out=torch.as_strided(torch.zeros(64), (1, 10), (3, 1)),
                residual=torch.as_strided(torch.zeros(64), (1, 10), (1, 1)))
    assert a.m == 1 and a.x_row % 4 == 0
    flat = torch.zeros(5000, dtype=BF16)
    kv = S.paged_struct(torch.as_strided(flat, (1, 1, 16, 64), (3, 5, 64, 1)), torch.as_strided(flat[2048:], (1, 1, 16, 64), (1024, 1024, 64, 1)),
                        _i32(3, 4), on_device=False)
    assert kv.page_stride % 8 == kv.head_stride % 8 == 0 and kv.slot_stride == 64
    for bad in (dict(k=torch.as_strided(odd, (3, 2, 64), (131, 64, 1))), dict(q=torch.as_strided(odd, (3, 4, 64), (257, 64, 1)))):
        with pytest.raises(ValueError, match="16 bytes"):
            _append(**bad)


def test_inputs_that_require_gradients():
    # there is no backward: a call that would record one is refused, one under no_grad is not
    def grad(t):
        return t.clone().requires_grad_()
    x = torch.zeros((3, 4, 64))
    calls = [(_append, dict(k=torch.zeros((3, 2, 64)))), (_append, dict(v=torch.zeros((3, 2, 64)))), (_append, dict(q=x)), (_append, dict(q_out=x)),
             (_append, dict(rope=torch.zeros((4, 32, 2)))), (_append, dict(q_norm=torch.zeros(64, dtype=BF16))),
             (_append, dict(k_norm=torch.zeros(64, dtype=BF16))), (_append, dict(k_cache=_cache()["k_cache"])), (_append, dict(v_cache=_cache()["v_cache"])),
             (_attention, dict(q=x)), (_attention, dict(out=x)), (_attention, dict(lse=torch.zeros((3, 4)))), (_attention, dict(v_cache=_cache()["v_cache"])),
             (_matvec, dict(x=torch.zeros((3, 128)))), (_matvec, dict(residual=torch.zeros((3, 10)))), (_matvec, dict(out=torch.zeros((3, 10)))),
             (_matvec, dict(scales=torch.zeros((10, 2), dtype=BF16)))]
    for f, kw in calls:
        with torch.no_grad():
            f(**{k: grad(v) for k, v in kw.items()})
        with torch.inference_mode():
            f(**{k: grad(v) for k, v in kw.items()})
        for t in (grad, lambda v: grad(v)[:]):              # a leaf, a view of one
            with pytest.raises(ValueError, match="%s.*gradient" % list(kw)[0]):
                f(**{k: t(v) for k, v in kw.items()})
    fp8 = torch.zeros((6, 2, 16, 64), dtype=E4M3)
    with pytest.raises(ValueError, match="gradient"):
        _attention(k_cache=fp8, v_cache=fp8, k_scale=torch.ones(2).requires_grad_(), v_scale=torch.ones(2))


def test_quantised_weights_of_a_parameter():
    w = torch.nn.Parameter(torch.randn((10, 128), generator=torch.Generator().manual_seed(0)))
    for zeros in (False, True):
        got = mk.quantize_q4(w, 64, zeros)
        assert not any(t.requires_grad for t in got)
        assert all(torch.equal(a, b) for a, b in zip(got, mk.quantize_q4(w.detach(), 64, zeros)))
        _matvec(codes=got[0], scales=got[1], zeros=got[2] if zeros else None)
