"""``matvec_q4`` against the products of its dequantised weights in 64 bits."""
import pytest
import torch

import serving_util as U

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")

BF16, F32 = torch.bfloat16, torch.float32


def _weights(n, k, group, zeros, seed=0):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.int32).to(torch.uint8)
    scales = ((torch.rand((n, k // group), generator=g) + 0.2) * 0.01).to(BF16)
    z = torch.randint(0, 16, (n, k // group), generator=g, dtype=torch.int32).to(torch.uint8) if zeros else None
    return codes, scales, z


def _check(y, x, w, residual, what):
    xd = x.to(U.F64)
    want = xd @ w.t()
    # a block's products: 16 chained sums at most; a multiply-add a block of 32 codes; the warps' and terms' sums
    err = (xd.abs() @ w.abs().t()) * ((16 + x.shape[1] / 32 + 32) * 2.0 ** -23)
    if residual is not None:
        want = want + residual.to(U.F64)
        err = err + (want.abs() + residual.to(U.F64).abs()) * 2.0 ** -24
    U.assert_within(y, want, U.half_step(x.dtype, want.abs() + err) + err, what)


def _run(m, n, k, group, x, zeros=False, residual=False, seed=0):
    codes, scales, z = _weights(n, k, group, zeros, seed)
    g = torch.Generator().manual_seed(seed + 1)
    xs = torch.randn((m, k), generator=g).to(x)
    res = torch.randn((m, n), generator=g).to(x) if residual else None
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    y = mk.matvec_q4(dev(xs), dev(codes), dev(scales), zeros=dev(z), residual=dev(res))
    torch.cuda.synchronize()
    _check(y, xs, U.dequantize(codes, scales, z), res, "matvec m %d n %d k %d group %d" % (m, n, k, group))


@pytest.mark.parametrize("x", [BF16, F32])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("m,n,k,group", [
    (1, 1, 32, 32), (1, 16, 64, 64), (1, 17, 128, 128), (1, 1000, 256, 128), (2, 33, 96, 32), (3, 100, 320, 64),
    (5, 250, 384, 128), (8, 64, 1024, 1024), (1, 4096, 1024, 64), (1, 100, 544, 32), (2, 700, 4160, 64),
    (3, 1203, 8192, 128), (4, 1100, 4096, 32), (9, 1203, 8192, 256), (1, 2400, 4224, 128), (3, 2048, 6144, 64), (8, 300, 2048, 32)])
def test_shapes(x, zeros, m, n, k, group):
    _run(m, n, k, group, x, zeros)


@pytest.mark.parametrize("m", [1, 2, 3, 5, 6, 8, 9, 10, 11, 16, 17, 32, 33, 70])
@pytest.mark.parametrize("x,group", [(BF16, 32), (BF16, 128), (F32, 64)])
def test_rows(m, x, group):
    _run(m, 131, 512, group, x, zeros=True, residual=True, seed=m)


@pytest.mark.parametrize("x", [BF16, F32])
def test_many_rounds_of_tiles(x):
    _run(1, 80013, 256, 64, x, residual=True)
    _run(9, 40011, 128, 32, x, zeros=True)


@pytest.mark.parametrize("m,x", [(1, F32), (2, F32), (7, BF16)])
def test_the_longest_rows(m, x):
    _run(m, 40, 32768, 128, x, seed=3)                      # fp32: one x row a pass


def test_strides_and_residual_in_place():
    codes, scales, z = _weights(96, 256, 64, True, seed=5)
    g = torch.Generator().manual_seed(6)
    x = torch.randn((4, 256), generator=g)
    wide = torch.zeros((4, 264), device="cuda")
    wide[:, 4:260] = x.cuda()
    out = torch.full((4, 101), 2.0, device="cuda")
    res = torch.randn((4, 96), generator=g)
    out[:, 3:99] = res.cuda()
    y = mk.matvec_q4(wide[:, 4:260], codes.cuda(), scales.cuda(), zeros=z.cuda(), residual=out[:, 3:99], out=out[:, 3:99])
    _check(y, x, U.dequantize(codes, scales, z), res, "in place")
    assert (out[:, :3] == 2).all() and (out[:, 99:] == 2).all()
    same = mk.matvec_q4(x[:1].cuda().expand(3, -1), codes.cuda(), scales.cuda(), zeros=z.cuda())
    assert torch.equal(same[0], same[1]) and torch.equal(same[0], same[2])


def test_infinities_and_nan_stay_in_their_rows():
    codes, scales, _ = _weights(64, 128, 32, False, seed=7)
    codes[:] = 0x9A                                         # codes 10 and 9: every weight is positive
    x = torch.ones((4, 128))
    x[1, 5], x[2, 6], x[3, 0] = float("inf"), float("nan"), 3.4e38
    y = mk.matvec_q4(x.cuda(), codes.cuda(), scales.cuda()).cpu()
    z = torch.ones((1, 128))
    z[0, 5], z[0, 9] = float("inf"), -1e30                  # finite values beside an infinity do not become one
    assert (mk.matvec_q4(z.cuda(), codes.cuda(), scales.cuda()) == float("inf")).all()
    assert torch.isfinite(y[0]).all() and (y[1] == float("inf")).all() and torch.isnan(y[2]).all() and torch.isfinite(y[3]).all()


@pytest.mark.parametrize("mag", [2.0 ** -90, 2.0 ** -20, 2.0 ** 80])
def test_rows_of_any_magnitude(mag):
    # a row is brought into fp16's range by a power of two: results do not depend on its size, nor on other rows'
    codes, scales, z = (t.cuda() for t in _weights(200, 512, 64, True, seed=11))
    x = torch.randn((3, 512), generator=torch.Generator().manual_seed(2)).cuda()
    want = mk.matvec_q4(x, codes, scales, zeros=z)
    x[1] *= mag
    got = mk.matvec_q4(x, codes, scales, zeros=z)
    got[1] /= mag
    assert torch.equal(got, want)


def test_nothing_to_do():
    codes, scales, _ = _weights(16, 64, 32, False)
    assert mk.matvec_q4(torch.zeros((0, 64), device="cuda"), codes.cuda(), scales.cuda()).shape == (0, 16)
    assert mk.matvec_q4(torch.zeros((2, 64), device="cuda"), codes[:0].cuda(), scales[:0].cuda()).shape == (2, 0)


def test_same_bits_on_streams_and_in_graphs():
    codes, scales, z = (t.cuda() for t in _weights(3000, 1024, 64, True, seed=8))
    x = torch.randn((4, 1024), generator=torch.Generator().manual_seed(1)).cuda()
    want = mk.matvec_q4(x, codes, scales, zeros=z)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [mk.matvec_q4(x, codes, scales, zeros=z, stream=s) for _ in range(3)]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        y = mk.matvec_q4(x, codes, scales, zeros=z)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        y.zero_()
    for t in got:
        assert torch.equal(t, want)


@pytest.mark.parametrize("zeros", [False, True])
def test_quantised_weights(zeros):
    w = torch.randn((64, 256), generator=torch.Generator().manual_seed(9)) * 0.02 + (0.01 if zeros else 0.0)
    q = [t.cuda() for t in mk.quantize_q4(w, 64, zeros)]
    x = torch.randn((2, 256), generator=torch.Generator().manual_seed(10))
    y = mk.matvec_q4(x.cuda(), q[0], q[1], zeros=q[2] if zeros else None)
    _check(y, x, U.dequantize(*q), None, "quantised")


# What is staged of x outweighs the weights: clusters of four CTAs with a slice of k each (fewer blocks than CTAs, blocks that
# do not divide by four, a broken last block, many tiles a cluster, several passes, one row of the longest k).
@pytest.mark.parametrize("x", [BF16, F32])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("m,n,k,group", [
    (100, 50, 256, 64), (200, 33, 128, 128), (60, 131, 416, 32), (40, 300, 640, 128), (30, 17, 1088, 64), (16, 2100, 4096, 128),
    (8, 2048, 6144, 32), (12, 5120, 5120, 64), (7, 16, 4480, 128), (33, 1000, 2944, 64)])
def test_slices_of_k(x, zeros, m, n, k, group):
    _run(m, n, k, group, x, zeros, residual=True, seed=21)


def test_slices_of_k_with_special_values():
    m, k = 48, 768
    codes, scales, _ = _weights(70, k, 32, False, seed=22)
    codes[:] = 0x9A                                         # every weight is positive
    x = torch.ones((m, k))
    x[1, 5], x[2, 700], x[3, 0], x[3, 767] = float("inf"), float("nan"), 3e38, -3e38
    x[4], x[5, :400], x[6, 200:] = 0.0, 0.0, 1e-30          # nothing at all, in some slices, next to nothing in others
    x[7, 3], x[7, 640] = float("inf"), -float("inf")
    w = U.dequantize(codes, scales)
    y = mk.matvec_q4(x.cuda(), codes.cuda(), scales.cuda()).cpu()
    assert (y[1] == float("inf")).all() and torch.isnan(y[2]).all() and torch.isnan(y[7]).all() and (y[4] == 0).all()
    rest = [0, 3, 5, 6] + list(range(8, m))
    _check(y[rest], x[rest], w, None, "rows beside the special ones")


def test_slices_of_k_same_bits_on_streams_and_in_graphs():
    codes, scales, z = (t.cuda() for t in _weights(900, 2048, 64, True, seed=23))
    x = torch.randn((20, 2048), generator=torch.Generator().manual_seed(24)).cuda()
    res = torch.randn((20, 900), generator=torch.Generator().manual_seed(25)).cuda()
    want = mk.matvec_q4(x, codes, scales, zeros=z, residual=res)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [mk.matvec_q4(x, codes, scales, zeros=z, residual=res, stream=s) for _ in range(3)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    y = torch.empty_like(res)
    with torch.cuda.graph(g):
        y.copy_(res)
        mk.matvec_q4(x, codes, scales, zeros=z, residual=y, out=y)   # in place
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    for t in got:
        assert torch.equal(t, want)
