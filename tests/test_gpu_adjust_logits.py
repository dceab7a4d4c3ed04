"""``adjust_logits`` against its definition in 64 bits."""
import math

import pytest
import torch

import prompt_util as P
import serving_util as U

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")

NAMES = ("tokens", "lengths", "prompts", "repetition", "presence", "frequency", "bias_ids", "bias", "mask")


def _inputs(n, v, columns, biases, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.rand(s, generator=g)  # noqa: E731
    a = dict(tokens=((v + 2) * r(n, columns) ** 3).int() - 1,        # -1 and v, v + 1 among them
             lengths=(r(n) * (columns + 1)).int(), repetition=r(n) + 0.6, presence=r(n) - 0.3, frequency=r(n) - 0.3,
             bias_ids=((v + 2) * r(n, biases)).int() - 1, bias=4 * r(n, biases) - 2,
             mask=torch.randint(-2 ** 31, 2 ** 31, (n, -(-v // 32)), generator=g).int())
    a["prompts"] = (a["lengths"] * r(n)).int()
    if n > 2:
        a["repetition"][1], a["presence"][1], a["frequency"][1] = 1.0, 0.0, 0.0
        a["mask"][2] = 0
    return a, torch.randn((n, v), generator=g) * 3


def _check(x, a, out=None, **kw):
    got = mk.adjust_logits(x, out=out, **{k: t.cuda() for k, t in a.items()}, **kw)
    want, err = P.adjusted(x.cpu() if out is not x else kw["before"], **a)
    U.assert_within(got, want, U.half_step(x.dtype, want) * (want.abs() < math.inf) + err, "logits")
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,v,columns,biases", [(1, 1, 1, 1), (1, 512, 40, 3), (3, 3001, 700, 20), (4, 33, 5, 40), (2, 20000, 17000, 5), (5, 4099, 300, 0)])
def test_all_together(dtype, n, v, columns, biases):
    a, x = _inputs(n, v, columns, biases)
    if not biases:
        del a["bias_ids"], a["bias"]
    _check(x.to(dtype).cuda(), a)


@pytest.mark.parametrize("which", [(), ("tokens", "repetition"), ("tokens", "lengths", "presence"), ("tokens", "lengths", "prompts", "frequency"),
                                   ("bias_ids", "bias"), ("mask",), ("tokens", "lengths", "mask")])
def test_each_alone(which):
    a, x = _inputs(3, 1003, 60, 9, seed=1)
    x = x.cuda()
    got = _check(x, {k: a[k] for k in which})
    if not which:
        assert torch.equal(got, x)


def test_rows_apart_in_place_and_padding():
    a, x = _inputs(5, 777, 50, 4, seed=2)
    a["lengths"][3] = -1
    for dtype, width, first in ((torch.float32, 781, 1), (torch.bfloat16, 800, 3), (torch.bfloat16, 777, 0)):
        wide = torch.zeros((5, width), dtype=dtype, device="cuda")
        view = wide[:, first:first + 777]
        view.copy_(x)
        ids, hist = torch.zeros((5, 9), dtype=torch.int32), torch.zeros((5, 61), dtype=torch.int32)
        ids[:, 2:6], hist[:, 5:55] = a["bias_ids"], a["tokens"]
        want, err = P.adjusted(view.cpu(), **a)
        want[3] = view[3].cpu().double()                      # left as it was
        b = {k: t.cuda() for k, t in a.items()}
        b["bias_ids"], b["tokens"] = ids.cuda()[:, 2:6], hist.cuda()[:, 5:55]
        tol = U.half_step(dtype, want) * (want.abs() < math.inf) + err
        other = torch.full((5, 784), 9.0, dtype=dtype, device="cuda")      # another alignment than the input's
        other[3, 2:779] = view[3]
        U.assert_within(mk.adjust_logits(view, out=other[:, 2:779], **b), want, tol, "logits elsewhere")
        assert (other[:, :2] == 9).all() and (other[:, 779:] == 9).all()
        assert mk.adjust_logits(view, out=view, **b) is view
        U.assert_within(view, want, tol, "logits in place")
        assert (wide[:, :first] == 0).all() and (wide[:, first + 777:] == 0).all()


def test_a_shared_mask_and_strange_numbers():
    a, x = _inputs(4, 300, 30, 6, seed=3)
    x[0, 5], x[1, 7], x[2, 9], x[3, 11] = math.inf, -math.inf, math.nan, 3e38
    a["tokens"][:, :4] = torch.tensor([5, 7, 9, 11], dtype=torch.int32)
    a["lengths"].clamp_(min=4)
    mask = torch.tensor([[-1] * 10], dtype=torch.int32)
    a["mask"] = mask.expand(4, -1)
    for dtype in (torch.float32, torch.bfloat16):
        y = x.to(dtype)
        got = mk.adjust_logits(y.cuda(), **{k: (t.cuda() if k != "mask" else mask.cuda().expand(4, -1)) for k, t in a.items()})
        want, err = P.adjusted(y, **a)
        want = torch.where(want.abs() > torch.finfo(dtype).max, want.sign() * math.inf, want)
        U.assert_within(got, want, torch.nan_to_num(U.half_step(dtype, want), posinf=0.0) + err, "logits")


def test_a_text_of_one_token():
    # as many as a 16-bit count holds, and more
    for columns in (16383, 16384, 40000):
        tokens = torch.full((1, columns), 3, dtype=torch.int32, device="cuda")
        got = mk.adjust_logits(torch.zeros((1, 8), device="cuda"), tokens=tokens, frequency=torch.ones(1, device="cuda"))
        assert got.tolist() == [[0.0, 0.0, 0.0, float(-columns), 0.0, 0.0, 0.0, 0.0]]


def test_nothing_to_do_and_a_captured_call():
    assert mk.adjust_logits(torch.zeros((0, 5), device="cuda")).shape == (0, 5)
    assert mk.adjust_logits(torch.zeros((3, 0), device="cuda")).shape == (3, 0)
    a, x = _inputs(8, 5000, 200, 3, seed=4)
    b, x = {k: t.cuda() for k, t in a.items()}, x.cuda()
    out = torch.zeros_like(x)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    mk.adjust_logits(x, out=out, stream=stream, **b)
    stream.synchronize()
    want = out.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mk.adjust_logits(x, out=out, **b)
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, want)
