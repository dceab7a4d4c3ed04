"""``quantize_fp8`` and ``matmul_fp8`` against their definitions in 64 bits."""
import math

import pytest
import torch

import prompt_util as P
import serving_util as U

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")

E4M3, BF16, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32


def _randn(*s, seed=0):
    return torch.randn(s, generator=torch.Generator().manual_seed(seed))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,k", [(1, 16), (1, 128), (3, 144), (5, 1024), (33, 6160), (700, 2048)])
def test_quantised_rows(dtype, m, k):
    x = (_randn(m, k, seed=m) * torch.exp2(torch.randint(-20, 20, (m, 1), generator=torch.Generator().manual_seed(k)).float())).to(dtype)
    x[0, :16] = 0.0
    codes, scales = mk.quantize_fp8(x.cuda())
    want, s = P.quantized(x)
    assert codes.dtype == E4M3 and codes.shape == (m, k) and scales.shape == s.shape
    assert torch.equal(scales.cpu().double(), s) and torch.equal(codes.cpu().double(), want)


def test_quantised_extremes():
    x = torch.zeros((6, 256))
    x[1, 3], x[2, 130], x[3, 0], x[4, 5], x[5, :128] = math.inf, math.nan, 3.3e38, 1e-42, -7.0
    x[1, 4], x[2, 131], x[3, 1] = 1.0, -2.0, 1.0
    codes, scales = (t.cpu().double() for t in mk.quantize_fp8(x.cuda()))
    assert math.isnan(codes[1, 3]) and codes[1, 4] == 0 and scales[1, 0] == math.inf and scales[1, 1] == 1
    assert math.isnan(codes[2, 130]) and codes[2, 131] == -448 and (codes[0] == 0).all() and (scales[0] == 1).all()
    assert codes[3, 0] == 448 and (codes[5, :128] == -448).all() and scales[5, 0] == torch.tensor(7.0).div(448).item()
    assert abs(codes[4, 5] * scales[4, 0]) <= 2e-42


def test_quantised_rows_apart():
    x = _randn(7, 300).to(BF16).cuda()[:, 8:296]
    codes, scales = torch.zeros((7, 320), device="cuda").to(E4M3)[:, 16:304], torch.zeros((7, 9), device="cuda")[:, 3:6]
    wide = torch.zeros((7, 304), dtype=BF16, device="cuda")
    wide[:, :288] = x
    got = mk.quantize_fp8(wide[:, :288], codes=codes, scales=scales)
    assert got[0] is codes and got[1] is scales
    want, s = P.quantized(x.cpu())
    assert torch.equal(codes.cpu().double(), want) and torch.equal(scales.cpu().double(), s)
    assert [t.shape for t in mk.quantize_fp8(torch.zeros((0, 32), device="cuda"))] == [(0, 32), (0, 1)]


def _operands(m, n, k, seed=0):
    x, xs = mk.quantize_fp8((_randn(m, k, seed=seed) * torch.exp2(_randn(m, 1, seed=seed + 1))).cuda())
    w, ws = mk.quantize_fp8_weight((_randn(n, k, seed=seed + 2) * 0.05).cuda())
    return x, xs, w, ws


# rows on either side of every choice of tile, odd columns, k that ends inside a block
@pytest.mark.parametrize("m,n,k", [(1, 1, 16), (1, 64, 128), (7, 300, 1040), (16, 4096, 1024), (17, 129, 256), (64, 257, 144), (65, 1000, 2048),
                                   (127, 2048, 512), (128, 128, 6144), (200, 777, 1024), (257, 513, 400), (777, 2048, 1024), (1500, 5000, 272)])
@pytest.mark.parametrize("dtype,residual", [(F32, True), (BF16, False)])
def test_products(m, n, k, dtype, residual):
    x, xs, w, ws = _operands(m, n, k)
    want, err = P.product(x.cpu(), xs.cpu(), w.cpu(), ws.cpu())
    r = None
    if residual:
        r = _randn(m, n, seed=9).to(dtype).cuda()
        want = want + r.cpu().double()
        err = err + want.abs() * 2.0 ** -24
    s = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mk.matmul_fp8(x, xs, w, ws, residual=r, dtype=dtype, status=s)
    assert got.dtype == dtype and int(s) == 0
    U.assert_within(got, want, U.half_step(dtype, want) + err, "product")
    again = mk.matmul_fp8(x, xs, w, ws, residual=r, dtype=dtype)
    assert torch.equal(got, again)


def test_strided_operands_in_place_and_types():
    m, n, k = 40, 200, 272
    x, xs, w, ws = _operands(m, n, k)
    xw, ww = torch.zeros((m, 320), device="cuda").to(E4M3), torch.zeros((n, 304), device="cuda").to(E4M3)
    xw[:, 16:288], ww[:, 32:304] = x, w
    xsw = torch.zeros((m, 7), device="cuda")
    xsw[:, 2:5] = xs
    out = torch.full((m, 203), 2.0, device="cuda")
    want, err = P.product(x.cpu(), xs.cpu(), w.cpu(), ws.cpu())
    got = mk.matmul_fp8(xw[:, 16:288], xsw[:, 2:5], ww[:, 32:304], ws, residual=out[:, 1:201], out=out[:, 1:201])
    U.assert_within(got, want + 2, U.half_step(F32, want + 2) + err + 2.0 ** -22, "product in place")
    assert (out[:, :1] == 2).all() and (out[:, 201:] == 2).all()
    assert mk.matmul_fp8(x, xs, w, ws).dtype == BF16
    assert mk.matmul_fp8(x, xs, w, ws, residual=out[:, :200]).dtype == F32
    assert mk.matmul_fp8(x[:0], xs[:0], w, ws).shape == (0, n) and mk.matmul_fp8(x, xs, w[:0], ws[:0]).shape == (m, 0)


def test_large_and_strange_values():
    # scales near fp32's ends, blocks that cancel, codes that are NaN
    m, n, k = 3, 130, 384
    x, w = torch.full((m, k), 448.0).to(E4M3).cuda(), torch.full((n, k), 448.0).to(E4M3).cuda()
    xs, ws = torch.tensor([[1e28, 1e-30, 0.0]] * m, device="cuda"), torch.tensor([[1e2, 1e-7, 1.0]] * 2, device="cuda")
    got = mk.matmul_fp8(x, xs, w, ws, dtype=F32)
    want, err = P.product(x.cpu(), xs.cpu(), w.cpu(), ws.cpu())
    U.assert_within(got, want, U.half_step(F32, want) + err, "large scales")
    x.view(torch.uint8)[1, 200] = 0x7F
    got = mk.matmul_fp8(x, xs, w, ws, dtype=F32)
    assert torch.isnan(got[1]).all() and torch.isfinite(got[0]).all() and torch.isfinite(got[2]).all()


@pytest.mark.parametrize("m,n,k", [(4, 1024, 1024), (300, 1000, 512)])
def test_captured_products(m, n, k):
    x, xs, w, ws = _operands(m, n, k)
    raw = _randn(m, k).bfloat16().cuda()
    out = torch.zeros((m, n), device="cuda", dtype=BF16)

    def step():
        return mk.matmul_fp8(*mk.quantize_fp8(raw), w, ws, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    raw.mul_(-3)
    g.replay()
    got = out.clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    q = mk.quantize_fp8(raw, stream=stream)
    mk.matmul_fp8(*q, w, ws, out=out, stream=stream)
    stream.synchronize()
    assert torch.equal(got, out) and got.abs().max() > 0
