"""``mk_attention_args`` as hosts have it that were built before ``sinks``: the same size and places (no GPU)."""
import ctypes as C
import os
import subprocess

import persistent_transformer_megakernel_gb300 as mk
from persistent_transformer_megakernel_gb300 import _binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


if not os.path.exists(mk.lib_path()):
    from persistent_transformer_megakernel_gb300 import build
    build.build()


class Before(C.Structure):
    _fields_ = [("n", C.c_int32), ("dtype", C.c_int32), ("n_q_heads", C.c_int32), ("q", C.c_void_p),
                ("out", C.c_void_p), ("q_row", C.c_int64), ("q_head", C.c_int64), ("out_row", C.c_int64),
                ("out_head", C.c_int64), ("lse", C.c_void_p), ("lengths", C.c_void_p), ("window", C.c_int32),
                ("scale", C.c_float), ("workspace", C.c_void_p), ("workspace_bytes", C.c_int64),
                ("status", C.c_void_p)]


def test_the_same_places():
    assert C.sizeof(B.mk_attention_args) == C.sizeof(Before)
    for name, _ in Before._fields_:
        assert getattr(B.mk_attention_args, name).offset == getattr(Before, name).offset, name


def test_the_headers_layout(tmp_path):
    # what the compiler makes of include/mk.h
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "mk.h"\nint main(void) { printf("%zu %zu %zu", sizeof(mk_attention_args), '
                   'offsetof(mk_attention_args, sinks), offsetof(mk_attention_args, status)); return 0; }\n')
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-I" + os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [C.sizeof(Before), B.mk_attention_args.sinks.offset, Before.status.offset]


def test_without_a_window_the_word_is_not_looked_at():
    lib = mk.load_library()
    kv = B.mk_paged_kv(16, 16, 1, 4, 2, 16, 64, 2048, 1024, 64, None, None, 16, 3, 4, 4)
    a = dict(n=0, dtype=0, n_q_heads=4, q=16, out=16, q_row=256, q_head=64, out_row=256, out_head=64, lengths=16, scale=0.125)
    call = lambda **f: lib.mk_paged_attention(C.byref(kv), C.byref(B.mk_attention_args(**{**a, **f})), None)  # noqa: E731
    assert call() == 0 and call(sinks=-7) == 0 and call(window=3, sinks=4) == 0 and call(window=3, sinks=-7) == -1
