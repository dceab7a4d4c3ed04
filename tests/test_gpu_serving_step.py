"""The serving operators together, as a decode step of several sequences uses
them: prompts prefilled by the framework's own decoder, their caches handed to a
paged one (``export_kv``), then every layer as 4-bit projections,
``paged_append``, ``paged_attention`` for all sequences at once -- against the
decoder's own steps of each sequence and its hidden states."""
import ctypes as C
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import workloads as W
from parity_util import assert_close

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")

MATRICES = ("wq", "wk", "wv", "wo", "w_gate", "w_up", "w_down")


def _q4_weights(s, seed=0):
    """Decoder weights whose matrices 4-bit codes hold exactly, and those codes and scales."""
    w = W.make_weights(s, seed)
    g = torch.Generator().manual_seed(seed + 1)
    packed = []
    for lw in w["layers"]:
        p = {}
        for name in MATRICES:
            n, k = lw[name].shape
            c = torch.randint(0, 16, (n, k), generator=g, dtype=torch.int32).to(torch.uint8)
            # scales of 2^-8 and 2^-7 by group: four-bit times a power of two is exact in bf16
            sc = torch.full((n, k // 64), 2.0 ** -8)
            sc[:, ::3] *= 2
            dense = (c.float() - 8) * sc.repeat_interleave(64, 1)
            lw[name] = dense.to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16).copy()
            p[name] = ((c[:, 0::2] | (c[:, 1::2] << 4)).contiguous().cuda(), sc.bfloat16().cuda())
        packed.append(p)
    return w, packed


def _bf16(bits):
    return torch.from_numpy(bits.view(np.int16).copy()).view(torch.bfloat16).cuda()


def _norm(x, gain, eps):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * gain.float()


@pytest.mark.parametrize("name,streams", [("gqa4", False), ("mrope_small", True), ("mrope_small_interleaved", True), ("mha", False)])
def test_batched_steps_follow_the_decoder(name, streams):
    s = W.shape(name)
    w, packed = _q4_weights(s)
    L, H, d, hq, hkv = s["n_layers"], s["hidden"], s["head_dim"], s["n_q_heads"], s["n_kv_heads"]
    prompts, steps, page = [1, 20, 37], 4, 12
    n = len(prompts)
    width = -(-(max(prompts) + steps) // page)
    order = np.random.default_rng(3).permutation(n * width + 2).astype(np.int32)
    table = torch.from_numpy(order[:n * width].reshape(n, width).copy()).cuda()
    caches = [[torch.zeros((n * width + 2, hkv, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(L)]

    # the decoder, one sequence at a time
    dec = mk.Decoder(s, w, max_seq=64)
    feeds, hidden = [], []
    for b, p in enumerate(prompts):
        dec.reset()
        ids = W.make_prompt(s["vocab_in"], p + steps, seed=5 + b)
        pos3 = torch.as_tensor(W.make_pos3(0, p + steps, distinct=True)).cuda() if streams else None
        dec.prefill(ids[:p], all_ids=False, pos3=None if pos3 is None else pos3[:, :p].contiguous())
        for l in range(L):
            dec.export_kv(l, *caches[l], table, seq=b)
        hid = torch.zeros((steps, L + 1, H), device="cuda")
        dec.decode(ids[p:], 0, hidden=hid, pos3=None if pos3 is None else pos3[:, p:].contiguous())
        feeds.append(torch.as_tensor(ids[p:]).cuda())
        hidden.append(hid)
    # refused: a range that is not there, other heads
    kv = mk.serving.paged_struct(*caches[0], table)
    lib = mk.load_library()
    stream = C.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert lib.mk_export_kv(dec.h, 0, 0, dec.position + 1, C.byref(kv), 0, 0, stream) == -1
    assert lib.mk_export_kv(dec.h, L, 0, 1, C.byref(kv), 0, 0, stream) == -1
    assert lib.mk_export_kv(dec.h, 0, 0, 1, C.byref(kv), n, 0, stream) == -1
    assert lib.mk_export_kv(dec.h, 0, 0, 1, C.byref(kv), 0, width * page, stream) == -10
    kv.n_kv_heads += 1
    assert lib.mk_export_kv(dec.h, 0, 0, 1, C.byref(kv), 0, 0, stream) == -2
    dec.close()

    # all sequences at once; padded to four rows, the last of them unused
    embed = _bf16(w["embed"])
    layers = [{k: _bf16(v) for k, v in lw.items() if k.endswith("norm")} for lw in w["layers"]]
    rope = mk.rope_table(256, d)
    table = torch.cat([table, torch.full_like(table[:1], -1)])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lengths = torch.tensor(prompts + [-1], dtype=torch.int32, device="cuda")
    for i in range(steps):
        slots = lengths.clone()
        lengths[:n] += 1
        positions = torch.stack([slots, slots + 7, 2 * slots + 3]).clamp_min(0).contiguous() if streams else None
        x = torch.zeros((n + 1, H), device="cuda")
        x[:n] = embed[torch.stack([f[i] for f in feeds]).long()].float()
        for l in range(L):
            p, lw = packed[l], layers[l]
            for b in range(n):
                assert_close(x[b].cpu().numpy(), hidden[b][i, l].cpu().numpy(), "%s step %d row %d layer %d" % (name, i, b, l))
            h = _norm(x, lw["attn_norm"], s["rms_eps"])
            q, k, v = (mk.matvec_q4(h, *p[m]).view(n + 1, -1, d) for m in ("wq", "wk", "wv"))
            q = mk.paged_append(k, v, *caches[l], table, slots, q=q, q_out=q, rope=rope, positions=positions,
                                mrope_sections=s["mrope_sections"], mrope_interleaved=bool(s.get("mrope_interleaved")),
                                q_norm=lw["q_norm"], k_norm=lw["k_norm"], eps=s["rms_eps"], status=status)
            o = torch.zeros_like(q)
            mk.paged_attention(q, *caches[l], table, lengths, out=o, status=status)
            x = mk.matvec_q4(o.view(n + 1, hq * d), *p["wo"], residual=x)
            h = _norm(x, lw["mlp_norm"], s["rms_eps"])
            gate, up = mk.matvec_q4(h, *p["w_gate"]), mk.matvec_q4(h, *p["w_up"])
            x = mk.matvec_q4(torch.nn.functional.silu(gate) * up, *p["w_down"], residual=x, out=x)
        for b in range(n):
            assert_close(x[b].cpu().numpy(), hidden[b][i, L].cpu().numpy(), "%s step %d row %d" % (name, i, b))
        assert (x[n] == 0).all()
    mk.check_status(status)


def test_exported_tokens_in_an_8_bit_cache():
    s = W.shape("tiny")
    dec = mk.Decoder(s, W.make_weights(s, 0), max_seq=64)
    dec.prefill(W.make_prompt(s["vocab_in"], 40, seed=1), all_ids=False)
    hkv, d = s["n_kv_heads"], s["head_dim"]
    table = torch.tensor([[7, 1, 4, 0]], dtype=torch.int32, device="cuda")
    kb, vb = (torch.zeros((8, hkv, 16, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dec.export_kv(1, kb, vb, table)
    k8, v8 = (torch.full((8, hkv, 16, d), 3.0, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = torch.tensor([0.02, 0.01], device="cuda"), torch.tensor([0.001, 0.002], device="cuda")
    dec.export_kv(1, k8, v8, table, first=5, count=30, slot=9, k_scale=ks, v_scale=vs)
    dec.close()
    for full, small, sc in ((kb, k8, ks), (vb, v8, vs)):
        a = full[table[0].long()].transpose(0, 1).reshape(hkv, 64, d)[:, 5:35].float()
        b = small.float()[table[0].long()].transpose(0, 1).reshape(hkv, 64, d)
        assert a.abs().max() > 0
        want = (a / sc[:, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn).float()
        assert torch.equal(b[:, 9:39], want)
        assert (b[:, :9] == 3).all() and (b[:, 39:] == 3).all()


def test_first_calls_inside_a_capture():
    # a new process whose first call of each operator is captured: nothing that a capture forbids happens there
    code = """
import torch
import persistent_transformer_megakernel_gb300 as mk
kc, vc = (torch.randn((8, 2, 16, 64), device="cuda").bfloat16() for _ in range(2))
table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
wide = torch.zeros((2, 4000), dtype=torch.int32, device="cuda")
n = torch.tensor([50, 7], dtype=torch.int32, device="cuda")
q = torch.randn((2, 4, 64), device="cuda")
codes, scales = torch.zeros((40, 64), dtype=torch.uint8, device="cuda"), torch.ones((40, 2), device="cuda").bfloat16()
x = torch.randn((2, 128), device="cuda")
torch.cuda.synchronize()
def step():
    k = mk.paged_append(q[:, :2], q[:, 2:], kc, vc, table, n, q=q)
    return [k, mk.paged_attention(k, kc, vc, table, n), mk.paged_attention(k, kc, vc, wide, n),
            mk.paged_attention(k[:1], kc, vc, table[:1], n[:1]), mk.matvec_q4(x, codes, scales)]
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
