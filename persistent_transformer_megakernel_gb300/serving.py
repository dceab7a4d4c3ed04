"""Operators of a decode step of several sequences: a paged KV cache and 4-bit weights.

``paged_append`` -> ``paged_attention`` over a page table, ``matvec_q4`` for
the projections, each one call of the C ABI (``include/mk.h``).  They enqueue on
the stream and return; what only the device can see (a page id outside the
cache, a position outside the rotary table) goes to an optional ``status`` word
that ``check_status`` turns into an ``MKError``.

The tensors of a call are checked here against what the kernels read and write,
as in ``_binding.check_options``: a wrong one is a ``ValueError``.
"""
from __future__ import annotations

import ctypes as C
from typing import Optional, Sequence, Tuple

import torch

from . import _binding as B

_TYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float8_e4m3fn: 2}
_workspaces: dict = {}      # bytes by (device, heads, kv heads, head_dim): sizes, no memory


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _vector(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, n: int, device) -> Optional[int]:
    """The address of a contiguous ``[n]`` tensor, or None."""
    if t is None:
        return None
    if t.dtype != dtype or t.dim() != 1 or t.shape[0] != n or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous tensor [%d] of dtype %s on %s" % (name, n, dtype, device))
    return t.data_ptr()


def _heads(t: torch.Tensor, name: str, n: int, d: int, dtype: torch.dtype, device, heads: int = 0) -> Tuple[int, int]:
    """Row and head strides of ``t`` [n][heads][d], its last dimension contiguous, the rest on 16-byte boundaries."""
    if t.dim() != 3 or t.dtype != dtype or t.device != device:
        raise ValueError("%s must be [rows][heads][head_dim] of dtype %s on %s" % (name, dtype, device))
    s, st = t.shape, t.stride()
    if s[0] != n or s[2] != d or (heads and s[1] != heads):
        raise ValueError("%s has shape %s; the call needs [%d][%s][%d]" % (name, tuple(s), n, heads or "heads", d))
    unit = 16 // t.element_size()
    if n and (st[2] != 1 or st[0] % unit or st[1] % unit or t.data_ptr() % 16):
        raise ValueError("%s: the last dimension must be contiguous and every row start on 16 bytes" % name)
    return st[0], st[1]


def paged_struct(k_cache: torch.Tensor, v_cache: torch.Tensor, table: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None, on_device: bool = True) -> B.mk_paged_kv:
    """The ``mk_paged_kv`` of a cache, checked: ``k_cache`` and ``v_cache``
    [n_pages][n_kv_heads][page_size][head_dim] of bf16 or float8_e4m3fn (equal
    strides, any order of the first three dimensions in memory), ``table`` int32
    [rows][pages], scales fp32 [n_kv_heads] for float8_e4m3fn only."""
    s, st = k_cache.shape, k_cache.stride()
    dev, dt = k_cache.device, k_cache.dtype
    _need(len(s) == 4 and dt in (torch.bfloat16, torch.float8_e4m3fn),
          "k_cache must be [n_pages][n_kv_heads][page_size][head_dim] of bf16 or float8_e4m3fn")
    _need(v_cache.shape == s and v_cache.stride() == st and v_cache.dtype == dt and v_cache.device == dev,
          "v_cache must have k_cache's shape, strides, dtype and device")
    _need(not on_device or k_cache.is_cuda, "the cache must be on a CUDA device")
    _need(s[3] in (64, 128), "head_dim must be 64 or 128")
    unit = 8 if dt == torch.bfloat16 else 16
    _need(s[0] > 0 and s[1] > 0 and s[2] > 0 and st[3] == 1 and st[0] % unit == 0 and st[1] % unit == 0 and st[2] % unit == 0
          and k_cache.data_ptr() % 16 == 0 and v_cache.data_ptr() % 16 == 0,
          "the cache's last dimension must be contiguous and every slot start on 16 bytes")
    _need(table.dim() == 2 and table.dtype == torch.int32 and table.device == dev
          and (table.stride(1) == 1 or table.shape[1] <= 1),
          "table must be int32 [rows][pages] on the cache's device, its rows contiguous")
    _need((k_scale is None) == (v_scale is None), "k_scale and v_scale go together")
    _need(k_scale is None or dt == torch.float8_e4m3fn, "scales are for a float8_e4m3fn cache")
    return B.mk_paged_kv(k_cache.data_ptr(), v_cache.data_ptr(), _TYPE[dt], s[0], s[1], s[2], s[3], st[0], st[1], st[2],
                         _vector(k_scale, "k_scale", torch.float32, s[1], dev),
                         _vector(v_scale, "v_scale", torch.float32, s[1], dev),
                         table.data_ptr(), table.shape[0], table.shape[1], table.stride(0))


def append_struct(kv: B.mk_paged_kv, k, v, slots, seqs, q, q_out, rope, positions, mrope_sections, mrope_interleaved,
                  q_norm, k_norm, eps, status) -> B.mk_append_args:
    """The checked ``mk_append_args`` of a ``paged_append`` call."""
    dev, dt, n, d = k.device, k.dtype, k.shape[0], kv.head_dim
    _need(dt in (torch.float32, torch.bfloat16), "k must be fp32 or bf16")
    a = B.mk_append_args()
    a.n, a.dtype = n, _TYPE[dt]
    a.k_row, a.k_head = _heads(k, "k", n, d, dt, dev, kv.n_kv_heads)
    a.v_row, a.v_head = _heads(v, "v", n, d, dt, dev, kv.n_kv_heads)
    a.k, a.v = k.data_ptr(), v.data_ptr()
    if q is not None:
        a.q_row, a.q_head = _heads(q, "q", n, d, dt, dev)
        a.n_q_heads = q.shape[1]
        a.out_row, a.out_head = _heads(q_out, "q_out", n, d, dt, dev, a.n_q_heads)
        a.q, a.q_out = q.data_ptr(), q_out.data_ptr()
    _need(slots is not None, "slots are needed")
    a.slots = _vector(slots, "slots", torch.int32, n, dev)
    if seqs is None:
        _need(n <= kv.table_rows, "without seqs, row i is sequence i: the table needs a row for each")
    else:
        a.seqs = _vector(seqs, "seqs", torch.int32, n, dev)
    if rope is not None:
        _need(rope.dim() == 3 and rope.shape[1:] == (d // 2, 2) and rope.dtype == torch.float32 and rope.is_contiguous()
              and rope.device == dev and rope.data_ptr() % 16 == 0, "rope must be the contiguous fp32 [rows][head_dim / 2][2] of rope_table")
        a.rope, a.rope_rows = rope.data_ptr(), rope.shape[0]
        if mrope_sections is not None:
            _need(len(mrope_sections) == 3 and min(mrope_sections) >= 0 and sum(mrope_sections) == d // 2,
                  "mrope_sections must be three counts that sum to head_dim / 2")
            _need(positions is not None and positions.shape == (3, n) and positions.dtype == torch.int32
                  and positions.device == dev and positions.is_contiguous(), "positions must be contiguous int32 [3][n] with mrope_sections")
            a.rope_mode = 2 if mrope_interleaved else 1
            a.mrope_sections[0], a.mrope_sections[1], a.mrope_sections[2] = mrope_sections
            a.positions = positions.data_ptr()
        elif positions is not None:
            a.positions = _vector(positions, "positions", torch.int32, n, dev)
    else:
        _need(positions is None and mrope_sections is None, "positions need a rope table")
    a.q_norm = _vector(q_norm, "q_norm", torch.bfloat16, d, dev)
    a.k_norm = _vector(k_norm, "k_norm", torch.bfloat16, d, dev)
    a.rms_eps = eps
    a.status = _vector(status, "status", torch.int32, 1, dev)
    return a


def _enqueue(fn, what: str, device, stream, *args) -> None:
    """One C call on ``device``'s current stream, or on ``stream``."""
    if device.index == torch.cuda.current_device():
        s = torch.cuda.current_stream(device) if stream is None else stream
        rc = fn(*args, s.cuda_stream)
    else:
        with torch.cuda.device(device):
            s = torch.cuda.current_stream(device) if stream is None else stream
            rc = fn(*args, s.cuda_stream)
    if rc:
        raise B.MKError(rc, what)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """Memory that belongs to the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def rope_table(rows: int, head_dim: int, theta: float = 1e6, device="cuda:0") -> torch.Tensor:
    """cos and sin of ``p * theta^(-2i / head_dim)`` for positions ``p < rows``,
    computed in double and rounded to fp32 [rows][head_dim / 2][2]."""
    w = theta ** (-2.0 * torch.arange(head_dim // 2, dtype=torch.float64) / head_dim)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * w
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous().to(device)


def paged_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, table: torch.Tensor,
                 slots: torch.Tensor, *, seqs: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                 q_out: Optional[torch.Tensor] = None, rope: Optional[torch.Tensor] = None,
                 positions: Optional[torch.Tensor] = None, mrope_sections: Optional[Sequence[int]] = None,
                 mrope_interleaved: bool = False, q_norm: Optional[torch.Tensor] = None,
                 k_norm: Optional[torch.Tensor] = None, eps: float = 1e-6, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None):
    """``mk_paged_append``: write ``k`` and ``v`` [n][kv heads][d] (fp32 or bf16, any
    row and head strides on 16 bytes) to their slots of the paged cache, with
    RMSNorm by the gains ``q_norm`` / ``k_norm`` and the rotation by ``rope`` on
    the way, and return the queries ``q`` treated alike (into ``q_out``, which may
    be ``q``; a new tensor by default; None without ``q``).

    ``slots`` int32 [n] are token indices in each row's sequence: row i of
    ``table``, or row ``seqs[i]``.  A negative slot marks a padding row: nothing
    of it is written, in ``q_out`` neither.  ``positions`` int32 [n] rotate by
    something else than the slot; with ``mrope_sections`` they are three streams
    [3][n] (``mrope_interleaved`` as ``rope_mode`` 2).  No two rows of a call may
    name the same slot of the cache."""
    kv = paged_struct(k_cache, v_cache, table, k_scale, v_scale)
    _need(k.device == k_cache.device, "k and the cache must be on the same device")
    if q is not None and q_out is None:
        q_out = _empty(q.shape, q.dtype, q.device, stream)
    a = append_struct(kv, k, v, slots, seqs, q, q_out, rope, positions, mrope_sections, mrope_interleaved, q_norm, k_norm,
                      eps, status)
    if a.n:
        _enqueue(B.load_library().mk_paged_append, "mk_paged_append", k.device, stream, C.byref(kv), C.byref(a))
    return q_out


def attention_struct(kv: B.mk_paged_kv, q, lengths, scale, window, out, lse, status) -> B.mk_attention_args:
    """The checked ``mk_attention_args`` of a ``paged_attention`` call, its workspace left open."""
    dev, dt, n, d = q.device, q.dtype, q.shape[0], kv.head_dim
    _need(dt in (torch.float32, torch.bfloat16), "q must be fp32 or bf16")
    a = B.mk_attention_args()
    a.n, a.dtype = n, _TYPE[dt]
    a.q_row, a.q_head = _heads(q, "q", n, d, dt, dev)
    hq = q.shape[1]
    _need(hq > 0 and hq % kv.n_kv_heads == 0, "q must have a multiple of the cache's %d heads" % kv.n_kv_heads)
    _need(n <= kv.table_rows, "the table has %d rows; the call needs %d" % (kv.table_rows, n))
    a.n_q_heads = hq
    a.out_row, a.out_head = _heads(out, "out", n, d, dt, dev, hq)
    a.q, a.out = q.data_ptr(), out.data_ptr()
    if lse is not None:
        _need(lse.shape == (n, hq) and lse.dtype == torch.float32 and lse.device == dev and lse.is_contiguous(),
              "lse must be a contiguous fp32 [%d][%d] on %s" % (n, hq, dev))
        a.lse = lse.data_ptr()
    _need(lengths is not None, "lengths are needed")
    a.lengths = _vector(lengths, "lengths", torch.int32, n, dev)
    _need(window >= 0, "window must be 0 (all) or the number of last tokens")
    a.window = window
    a.scale = d ** -0.5 if scale is None else scale
    a.status = _vector(status, "status", torch.int32, 1, dev)
    return a


def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, table: torch.Tensor, lengths: torch.Tensor,
                    *, scale: Optional[float] = None, window: int = 0, k_scale: Optional[torch.Tensor] = None,
                    v_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``mk_paged_attention``: attention of one new token per row, ``q`` [n][heads][d]
    (fp32 or bf16), over the first ``lengths[i]`` (the last ``window`` of them,
    if not 0) tokens of ``table``'s row i.  Returns ``out`` like ``q`` (it may be
    ``q``); ``lse`` fp32 [n][heads] receives the log of each softmax's sum.  A row
    of length 0 gives zeros and -inf, one of negative length is left as it was."""
    kv = paged_struct(k_cache, v_cache, table, k_scale, v_scale)
    _need(q.device == k_cache.device, "q and the cache must be on the same device")
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    a = attention_struct(kv, q, lengths, scale, window, out, lse, status)
    if a.n == 0:
        return out
    lib = B.load_library()
    key = (q.device.index, a.n_q_heads, kv.n_kv_heads, kv.head_dim)
    size = _workspaces.get(key)
    if size is None:
        with torch.cuda.device(q.device):
            size = lib.mk_paged_attention_workspace(*key[1:])
        if size < 0:
            raise B.MKError(size, "mk_paged_attention_workspace")
        _workspaces[key] = size
    ws = _empty(size, torch.uint8, q.device, stream)
    a.workspace, a.workspace_bytes = ws.data_ptr(), size
    _enqueue(lib.mk_paged_attention, "mk_paged_attention", q.device, stream, C.byref(kv), C.byref(a))
    return out


def matvec_struct(x, codes, scales, zeros, residual, y) -> B.mk_matvec_q4_args:
    """The checked ``mk_matvec_q4_args`` of a ``matvec_q4`` call."""
    dev, dt = x.device, x.dtype
    _need(x.dim() == 2 and dt in (torch.float32, torch.bfloat16), "x must be [rows][k] of fp32 or bf16")
    m, k = x.shape
    _need(codes.dim() == 2 and codes.shape[1] * 2 == k and codes.dtype == torch.uint8 and codes.is_contiguous() and codes.device == dev,
          "codes must be contiguous uint8 [n][k / 2] on %s" % dev)
    n = codes.shape[0]
    _need(scales.dim() == 2 and scales.shape[0] == n and scales.dtype == torch.bfloat16 and scales.is_contiguous() and scales.device == dev
          and 0 < scales.shape[1] and k % scales.shape[1] == 0 and k > 0, "scales must be contiguous bf16 [n][k / group] on %s" % dev)
    group = k // scales.shape[1]
    _need(group in (32, 64) or group % 128 == 0, "the group must be 32, 64 or a multiple of 128")
    _need(zeros is None or (zeros.shape == scales.shape and zeros.dtype == torch.uint8 and zeros.is_contiguous() and zeros.device == dev),
          "zeros must be contiguous uint8 of scales' shape")
    unit = 4 if dt == torch.float32 else 8
    _need(not m or (x.stride(1) == 1 and x.stride(0) % unit == 0 and x.data_ptr() % 16 == 0),
          "x's last dimension must be contiguous and every row start on 16 bytes")
    _need(codes.data_ptr() % 16 == 0, "codes must start on 16 bytes")
    for t, name in ((residual, "residual"), (y, "out")):
        _need(t is None or (t.shape == (m, n) and t.dtype == dt and t.device == dev and (t.stride(1) == 1 or n <= 1)),
              "%s must be [%d][%d] of dtype %s on %s, its rows contiguous" % (name, m, n, dt, dev))
    a = B.mk_matvec_q4_args(m, n, k, group, _TYPE[dt], x.data_ptr(), x.stride(0), codes.data_ptr(), scales.data_ptr(),
                            None if zeros is None else zeros.data_ptr(), None, 0, y.data_ptr(), y.stride(0))
    if residual is not None:
        a.residual, a.residual_row = residual.data_ptr(), residual.stride(0)
    return a


def matvec_q4(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, *, zeros: Optional[torch.Tensor] = None,
              residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``mk_matvec_q4``: ``x`` [rows][k] (fp32 or bf16) times the transpose of the
    4-bit weights of ``quantize_q4``, plus ``residual`` [rows][n] (which may be
    ``out``).  ``codes`` uint8 [n][k / 2], ``scales`` bf16 and ``zeros`` uint8 (8
    everywhere if None) [n][k / group]."""
    _need(x.is_cuda and x.dim() == 2 and codes.dim() == 2, "x [rows][k] and codes [n][k / 2] must be on a CUDA device")
    if out is None:
        out = _empty((x.shape[0], codes.shape[0]), x.dtype, x.device, stream)
    a = matvec_struct(x, codes, scales, zeros, residual, out)
    if a.m and a.n:
        _enqueue(B.load_library().mk_matvec_q4, "mk_matvec_q4", x.device, stream, C.byref(a))
    return out


def quantize_q4(w: torch.Tensor, group: int = 64, zeros: bool = False):
    """4-bit codes of ``w`` [n][k], once per weight: ``(codes uint8 [n][k / 2], scales
    bf16 [n][k / group])`` with codes 0 .. 15 around 8, or, with ``zeros``, a zero
    point of each group as a third tensor (uint8), which uses all 16 codes of a
    group that is not centred.  Codes are the nearest to w over the rounded scale."""
    n, k = w.shape
    _need(group in (32, 64) or (group > 0 and group % 128 == 0), "the group must be 32, 64 or a multiple of 128")
    _need(k % group == 0, "the group must divide k")
    x = w.float().view(n, k // group, group)
    if zeros:
        lo, hi = x.amin(-1).clamp_max(0.0), x.amax(-1).clamp_min(0.0)
        scale = ((hi - lo) / 15.0).bfloat16()
    else:
        scale = (x.abs().amax(-1) / 7.0).bfloat16()
    s = scale.float()
    s = torch.where(s > 0, s, torch.ones_like(s))[..., None]
    zero = (-lo[..., None] / s).round().clamp(0, 15) if zeros else torch.full_like(s, 8.0)
    c = ((x / s).round() + zero).clamp(0, 15).to(torch.uint8).view(n, k)
    codes = (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous()
    if zeros:
        return codes, scale, zero[..., 0].to(torch.uint8)
    return codes, scale


def check_status(status: torch.Tensor) -> None:
    """Wait for and raise the error that a paged operator has left in ``status``
    (int32 [1], zeroed before the call); nothing if there is none."""
    code = int(status.item())
    if code:
        raise B.MKError(code, "paged operator")
