"""Operators of a step of several sequences: a paged KV cache, 4-bit and 8-bit weights.

``paged_plan`` gives a step's tokens their rows, slots and pages;
``paged_append`` -> ``paged_attention`` (single tokens) or
``paged_prompt_attention`` (prompts) over a page table; ``matvec_q4`` (few
rows) or ``quantize_fp8`` -> ``matmul_fp8`` (many) for the projections;
``adjust_logits`` before a token is chosen.  Each is one call of the C ABI
(``include/mk.h``).  They enqueue on the stream and return; what only the device can see (a page id outside the
cache, a position outside the rotary table) goes to an optional ``status`` word
that ``check_status`` turns into an ``MKError``.  They have no gradients:
a tensor that requires them is refused unless gradients are off
(``torch.no_grad``), and so is one that carries a tangent of forward-mode
differentiation.

They are functions of the module ``_mktorch`` (``csrc/mk_torch.cpp``,
``csrc/mk_torch_prompts.h``), which checks the tensors of a call against what
the kernels read and write (a wrong one is a ``ValueError``).  It is loaded when the first of them is asked for, and
like the library it must have been built.
"""
from __future__ import annotations

import importlib
import os
from typing import Optional

import torch

from . import _binding as B

NATIVE = ("paged_append", "paged_attention", "matvec_q4", "paged_plan", "paged_prompt_attention", "quantize_fp8", "matmul_fp8",
          "adjust_logits")


def native():
    """The module ``_mktorch``.  Raises if it is not built."""
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_mktorch.so")
    if not os.path.exists(path):
        raise RuntimeError("_mktorch.so not built at %s: run __graft_entry__.build()" % path)
    B.load_library()
    return importlib.import_module("._mktorch", __package__)


def __getattr__(name: str):
    if name not in NATIVE:
        raise AttributeError("module %r has no attribute %r" % (__name__, name))
    f = getattr(native(), name)
    globals()[name] = f
    return f


def paged_struct(k_cache: torch.Tensor, v_cache: torch.Tensor, table: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None, on_device: bool = True) -> B.mk_paged_kv:
    """The ``mk_paged_kv`` of a cache, its tensors checked as ``paged_append`` does."""
    return B.mk_paged_kv.from_buffer_copy(native().paged_kv(k_cache, v_cache, table, k_scale=k_scale, v_scale=v_scale, on_device=on_device))


def rope_table(rows: int, head_dim: int, theta: float = 1e6, device="cuda:0") -> torch.Tensor:
    """cos and sin of ``p * theta^(-2i / head_dim)`` for positions ``p < rows``,
    computed in double and rounded to fp32 [rows][head_dim / 2][2]."""
    w = theta ** (-2.0 * torch.arange(head_dim // 2, dtype=torch.float64) / head_dim)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * w
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous().to(device)


def quantize_q4(w: torch.Tensor, group: int = 64, zeros: bool = False):
    """4-bit codes of ``w`` [n][k], once per weight: ``(codes uint8 [n][k / 2], scales
    bf16 [n][k / group])`` with codes 0 .. 15 around 8, or, with ``zeros``, a zero
    point of each group as a third tensor (uint8), which uses all 16 codes of a
    group that is not centred.  Codes are the nearest to w over the rounded scale."""
    w = w.detach()
    n, k = w.shape
    if not (group in (32, 64) or (group > 0 and group % 128 == 0)) or k % group:
        raise ValueError("the group must be 32, 64 or a multiple of 128, and divide k (%d)" % k)
    x = w.float().reshape(n, k // group, group)
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


def quantize_fp8_weight(w: torch.Tensor):
    """8-bit codes of ``w`` [n][k] (k a multiple of 16), once per weight: ``(codes
    float8_e4m3fn [n][k], scales fp32 [n / 128][k / 128], rounded up)``; a block of
    128 x 128 has the scale largest / 448.  NaN stays NaN and does not count for
    the scale."""
    w = w.detach()
    n, k = w.shape
    if k % 16 or k == 0:
        raise ValueError("k (%d) must be a multiple of 16" % k)
    nb, kb = -(-n // 128), -(-k // 128)
    x = torch.nn.functional.pad(w.float(), (0, kb * 128 - k, 0, nb * 128 - n)).view(nb, 128, kb, 128)
    largest = x.abs().nan_to_num_(nan=0.0, posinf=float("inf")).amax((1, 3))
    scales = largest / torch.full_like(largest, 448.0)
    scales = torch.where(scales > 0, scales, torch.ones_like(scales))
    codes = (x / scales[:, None, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(nb * 128, kb * 128)[:n, :k]
    return codes.contiguous(), scales


def check_status(status: torch.Tensor, stream=None) -> None:
    """Wait for and raise the error that a paged operator has left in ``status``
    (int32 [1], zeroed before the call); nothing if there is none.  ``stream`` is
    the operator's, where that was not the current one."""
    if stream is None:
        code = int(status.item())
    else:
        with torch.cuda.stream(stream):                  # the word is copied, and waited for, behind the operator
            code = int(status.item())
    if code:
        raise B.MKError(code, "paged operator")
