"""The operators together, as a batch's prompts and the steps behind them use them: a plan of rows, slots and pages, 8-bit
projections, the paged cache, attention under a window with first tokens, adjusted logits.  Each operator's result is
compared with its definition in 64 bits on the inputs it got; pages and tokens are followed by the test itself."""
import numpy as np
import pytest
import torch

import prompt_util as P
import serving_util as U

pytestmark = pytest.mark.gpu

mk = pytest.importorskip("persistent_transformer_megakernel_gb300")

BF16, F32 = torch.bfloat16, torch.float32
H, HQ, HKV, D, INNER, VOCAB, LAYERS, PAGE, WINDOW, SINKS, EPS = 256, 4, 2, 64, 400, 1003, 2, 12, 40, 3, 1e-6
WIDTH, PAGES = 12, 60


def _weights():
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    w = dict(embed=r(VOCAB, H).to(BF16).cuda(), head=mk.quantize_fp8_weight((r(VOCAB, H) * H ** -0.5).cuda()), layers=[])
    for _ in range(LAYERS):
        w["layers"].append({n: mk.quantize_fp8_weight((r(o, i) * i ** -0.5).cuda()) for n, o, i in
                            (("qkv", (HQ + 2 * HKV) * D, H), ("o", H, HQ * D), ("up", 2 * INNER, H), ("down", H, INNER))})
        w["layers"][-1]["norms"] = [(1 + 0.1 * r(D)).to(BF16).cuda() for _ in range(2)]
    return w


def _norm(x):
    x = x.float()
    return (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)).to(BF16)


class Run:
    """One model's pass over token rows; ``check``: each operator next to its definition."""

    def __init__(self, check):
        self.check = check
        self.w = _weights()
        self.cache = [[torch.zeros((PAGES, HKV, PAGE, D), dtype=BF16, device="cuda") for _ in range(2)] for _ in range(LAYERS)]
        self.rope = mk.rope_table(WIDTH * PAGE, D)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def product(self, x, name, weights, residual=None, dtype=BF16):
        codes, scales = mk.quantize_fp8(x)
        y = mk.matmul_fp8(codes, scales, *weights, residual=residual, dtype=dtype, status=self.status)
        if self.check:
            want, s = P.quantized(x.cpu())
            assert torch.equal(codes.cpu().double(), want) and torch.equal(scales.cpu().double(), s)
            want, err = P.product(codes.cpu(), scales.cpu(), *(t.cpu() for t in weights))
            if residual is not None:
                want = want + residual.cpu().double()
                err = err + want.abs() * 2.0 ** -24
            U.assert_within(y, want, U.half_step(dtype, want) + err, name)
        return y

    def layers(self, ids, attend, table, seqs, slots):
        x = self.w["embed"][ids.long()]
        for l, w in enumerate(self.w["layers"]):
            qkv = self.product(_norm(x), "qkv", w["qkv"]).view(-1, HQ + 2 * HKV, D)
            before = [c.clone() for c in self.cache[l]] if self.check else None
            q = mk.paged_append(qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], *self.cache[l], table, slots, seqs=seqs, q=qkv[:, :HQ], rope=self.rope,
                                q_norm=w["norms"][0], k_norm=w["norms"][1], eps=EPS, status=self.status)
            if self.check:
                self.appended(qkv, q, l, before, table, seqs, slots)
            a = attend(q, l, table)
            x = self.product(a.view(-1, HQ * D), "o", w["o"], residual=x)
            h = self.product(_norm(x), "up", w["up"])
            x = self.product(torch.nn.functional.silu(h[:, :INNER]) * h[:, INNER:], "down", w["down"], residual=x)
        return x

    def appended(self, qkv, q, l, before, table, seqs, slots):
        live = (slots >= 0).nonzero()[:, 0].cpu()
        p, s = slots.cpu()[live].long(), seqs.cpu()[live].long()
        angle = U.rotary(p, D)
        n = self.w["layers"][l]["norms"]
        for got, want in ((q.cpu()[live], U.turned(qkv[:, :HQ].cpu()[live], n[0].cpu(), angle, EPS)),
                          (self.cache[l][0].cpu()[table.cpu()[s, p // PAGE].long(), :, p % PAGE], U.turned(qkv[:, HQ:HQ + HKV].cpu()[live], n[1].cpu(), angle, EPS)),
                          (self.cache[l][1].cpu()[table.cpu()[s, p // PAGE].long(), :, p % PAGE], U.turned(qkv[:, HQ + HKV:].cpu()[live], None, None, EPS))):
            U.assert_within(got, want[0], U.half_step(BF16, want[0]) + want[1], "appended")
        for now, old in zip(self.cache[l], before):
            old[table[seqs[live].long(), (slots[live] // PAGE).long()].long(), :, (slots[live] % PAGE).long()] = \
                now[table[seqs[live].long(), (slots[live] // PAGE).long()].long(), :, (slots[live] % PAGE).long()]
            assert torch.equal(now, old)                      # nothing else was written

    def next_ids(self, x, a):
        logits = self.product(_norm(x), "head", self.w["head"], dtype=F32)
        y = mk.adjust_logits(logits, **a)
        if self.check:
            want, err = P.adjusted(logits.cpu(), **{k: v.cpu() for k, v in a.items()})
            live = a["lengths"].cpu() >= 0
            U.assert_within(y.cpu()[live], want[live], (U.half_step(F32, want) * (want.abs() < 1e30) + err)[live], "logits")
        return y.argmax(-1).int()


def _params(n, g):
    return dict(repetition=1 + torch.rand(n, generator=g), presence=torch.rand(n, generator=g), frequency=torch.rand(n, generator=g),
                bias_ids=torch.randint(0, VOCAB, (n, 5), generator=g).int(), bias=torch.randn((n, 5), generator=g),
                mask=torch.randint(-2 ** 31, 2 ** 31, (n, -(-VOCAB // 32)), generator=g).int())


@pytest.mark.parametrize("check", [True, False])
def test_prompts_and_the_steps_behind_them(check):
    g = torch.Generator().manual_seed(1)
    n, counts, steps = 4, [50, 1, 0, 17], 6
    lengths = torch.tensor([0, 0, -1, 0], dtype=torch.int32, device="cuda")
    run = Run(check)
    table = torch.full((n, WIDTH), -1, dtype=torch.int32, device="cuda")
    free = torch.from_numpy(np.random.default_rng(0).permutation(PAGES).astype("int32")).cuda()
    used = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = 80                                                  # of which 68 are in use
    texts = [torch.randint(0, VOCAB, (c,), generator=g).int() for c in counts]
    params = {k: v.cuda() for k, v in _params(n, g).items()}
    tokens = torch.zeros((n, 100), dtype=torch.int32, device="cuda")
    for i, t in enumerate(texts):
        tokens[i, :counts[i]] = t.cuda()
    prompts = torch.tensor(counts, dtype=torch.int32, device="cuda")

    # the prompts, in two chunks
    done = [0] * n
    last = torch.zeros((n, H), dtype=BF16, device="cuda")
    for part in (0.4, 1.0):
        now = [int(c * part) - d for c, d in zip(counts, done)]
        seqs, slots, starts, lengths, used = mk.paged_plan(lengths, table, free, used, PAGE, counts=torch.tensor(now, dtype=torch.int32).cuda(), rows=rows,
                                                           status=run.status)
        assert slots.tolist() == [p for d, c in zip(done, now) for p in range(d, d + c)] + [-1] * (rows - sum(now))
        ids = torch.zeros(rows, dtype=torch.int32, device="cuda")
        ids[:sum(now)] = torch.cat([t[d:d + c] for t, d, c in zip(texts, done, now)]).cuda()

        def attend(q, l, table):
            out = mk.paged_prompt_attention(q, *run.cache[l], table, starts, lengths, window=WINDOW, sinks=SINKS, out=torch.zeros_like(q), status=run.status)
            if check:
                want, _, err, _ = P.prompt_attention(q.cpu(), *(c.cpu() for c in run.cache[l]), table.cpu(), starts.cpu(), lengths.cpu(), D ** -0.5, WINDOW, SINKS)
                k = int(starts[-1])
                U.assert_within(out[:k], want[:k], (U.half_step(BF16, want) + err)[:k], "prompt")
                assert (out[k:] == 0).all()
            return out
        x = run.layers(ids, attend, table, seqs, slots)
        done = [d + c for d, c in zip(done, now)]
        for i in range(n):
            if now[i]:
                last[i] = x[int(starts[i + 1]) - 1]
    hist = torch.tensor([50, 1, -1, 17], dtype=torch.int32, device="cuda")
    ids = run.next_ids(last, dict(params, tokens=tokens, lengths=hist, prompts=prompts))

    # the steps: a token a sequence, the third row unused; captured once where nothing is checked
    state = dict(ids=ids.clone(), lengths=lengths.clone(), used=used.clone(), hist=hist.clone())
    made = torch.zeros((steps, n), dtype=torch.int32, device="cuda")
    at = torch.arange(n, device="cuda")
    live = hist >= 0

    def step():
        s = state
        tokens[at[live], s["hist"][live].long()] = s["ids"][live]
        s["hist"].add_(live.int())
        seqs, slots, starts, totals, _ = mk.paged_plan(s["lengths"], table, free, s["used"], PAGE, totals=s["lengths"], used_out=s["used"], status=run.status)

        def attend(q, l, table):
            out = mk.paged_attention(q, *run.cache[l], table, totals, window=WINDOW, sinks=SINKS, out=torch.zeros_like(q), status=run.status)
            if check:
                want, _, err, _ = P.prompt_attention(q.cpu(), *(c.cpu() for c in run.cache[l]), table.cpu(), starts.cpu(), totals.cpu(), D ** -0.5, WINDOW, SINKS)
                U.assert_within(out[live], want[live.cpu()], (U.half_step(BF16, want) + err)[live.cpu()], "token")
                assert (out[2] == 0).all()
            return out
        x = run.layers(s["ids"].clamp_min(0), attend, table, seqs, slots)
        s["ids"].copy_(run.next_ids(x, dict(params, tokens=tokens, lengths=s["hist"], prompts=prompts)))
    if check:
        for i in range(steps):
            step()
            made[i] = state["ids"]
    else:
        live_rows = live.nonzero()[:, 0]
        live = live_rows                                       # (no shapes that depend on data inside a capture)
        keep = {k: v.clone() for k, v in state.items()}
        kept = tokens.clone(), table.clone()

        def again():
            for k, v in keep.items():
                state[k].copy_(v)
            tokens.copy_(kept[0]), table.copy_(kept[1])
        mask = (hist >= 0).int()

        def captured_step():
            s = state
            tokens.scatter_(1, s["hist"].clamp_min(0).long()[:, None], torch.where(mask[:, None] > 0, s["ids"][:, None], tokens.gather(1, s["hist"].clamp_min(0).long()[:, None])))
            s["hist"].add_(mask)
            seqs, slots, _, totals, _ = mk.paged_plan(s["lengths"], table, free, s["used"], PAGE, totals=s["lengths"], used_out=s["used"], status=run.status)
            x = run.layers(s["ids"].clamp_min(0), lambda q, l, t: mk.paged_attention(q, *run.cache[l], t, totals, window=WINDOW, sinks=SINKS,
                                                                                     out=torch.zeros_like(q), status=run.status), table, seqs, slots)
            s["ids"].copy_(run.next_ids(x, dict(params, tokens=tokens, lengths=s["hist"], prompts=prompts)))
        plain = []
        for _ in range(steps):
            captured_step()
            plain.append(state["ids"][live_rows].clone())
        again()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured_step()
        again()
        for i in range(steps):
            graph.replay()
            assert torch.equal(state["ids"][live_rows], plain[i])
    mk.check_status(run.status)
    assert state["lengths"].tolist() == [50 + steps, 1 + steps, -1, 17 + steps]
    assert int(state["used"]) == sum(-(-(c + steps) // PAGE) for c in (50, 1, 17))
    pages = table[table >= 0].tolist()
    assert len(pages) == len(set(pages)) == int(state["used"])
