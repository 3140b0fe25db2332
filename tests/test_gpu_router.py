"""muon_router_balance and muon_router_bias_step against the definition in 64 bits: expert numbers, score forms, packed
sequences (empty ones, gaps, tokens of none), masks, dropped and repeated choices, rows without a score, strides.

Tolerances.  Counts and biases are exact.  A probability is off by the exponent's rounding (a product with log2 e, 2^-24 of
an exponent below 16 in what counts: 2^-20), the sum's (log2 E + 8 additions: 2^-20) and a few more of 2^-23, 2^-18 in all;
a gradient has that twice and the factor's, relative to p_i (|c_i - mean| + sum_j p_j |c_j - mean|) q_i, which bounds its
terms: 2^-16 of that, and half a step of its own type.  The loss, sums of positive terms: 2^-17."""

import numpy as np
import pytest

import muon_step_amd as ms
from gpu_util import say

pytestmark = pytest.mark.gpu

COEF = 1e-2


@pytest.fixture(scope="module")
def ctx():
    c = ms.Context(0)
    yield c
    c.close()


def oracle(x, chosen, offsets, mask, score, scale=1.0):
    """(loss, counts, gradient, bound of the gradient's terms, rows that are written) in 64 bits, token by token."""
    tokens, experts = x.shape
    top = chosen.shape[1]
    with np.errstate(all="ignore"):
        x = x.astype(np.float64)
        z = x if score == "softmax" else -np.logaddexp(0.0, -x)
        m = np.max(z, axis=1, keepdims=True)
        w = np.where(np.isneginf(z), 0.0, np.exp(z - np.where(np.isneginf(m), 0.0, m)))
        total = w.sum(1, keepdims=True)
        p = np.where(total == 0, 0.0, w / np.where(total == 0, 1.0, total))
        q = np.ones_like(x) if score == "softmax" else np.exp(-np.logaddexp(0.0, x))
    counts = np.zeros(experts, np.int64)
    grad, bound = np.zeros((tokens, experts)), np.zeros((tokens, experts))
    written = np.zeros(tokens, bool)
    spans = [(max(0, a), min(tokens, b)) for a, b in zip(offsets, offsets[1:])]
    taking = [[t for t in range(a, b) if mask[t]] for a, b in spans]
    live = sum(1 for rows in taking if rows)
    loss = 0.0
    for (a, b), rows in zip(spans, taking):
        written[a:max(a, b)] = True
        if not rows:
            continue
        picks = chosen[rows].ravel()
        picks = picks[(picks >= 0) & (picks < experts)]
        c = np.bincount(picks, minlength=experts)
        counts += c
        f = COEF / live * experts * c / (top * len(rows)) / len(rows)
        loss += float((p[rows] * f).sum())
        # a row's probabilities sum to 1 (or are all 0): the factors' mean drops out of the gradient, in whole numbers, so
        # that even loads give exactly none here too
        away = COEF / live * (experts * c - c.sum()) / (top * len(rows)) / len(rows)
        grad[rows] = scale * p[rows] * (away - (p[rows] * away).sum(1, keepdims=True)) * q[rows]
        bound[rows] = scale * p[rows] * (np.abs(away) + (p[rows] * np.abs(away)).sum(1, keepdims=True)) * q[rows]
    return loss, counts, grad, bound, written


class Batch:
    def __init__(self, rng, tokens, experts, top, offsets=None, score="softmax", dtype="f32", bits=64, mask=False, gap=0,
                 drop=0.0, logits=None):
        import torch
        self.score, self.gap, self.experts = score, gap, experts
        x = rng.standard_normal((tokens, experts)) + rng.standard_normal(experts) * 0.5 if logits is None else logits
        full = rng.standard_normal((tokens, experts + gap))
        full[:, :experts] = x
        kind = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.full = torch.from_numpy(full.astype(np.float32)).to(kind).cuda()
        self.x = self.full[:, :experts].float().cpu().numpy()
        self.chosen = rng.integers(0, experts, (tokens, top))
        if drop:
            self.chosen[rng.random((tokens, top)) < drop] = -1
            self.chosen[rng.random((tokens, top)) < drop / 4] = experts + 3
        self.offsets = [0, tokens] if offsets is None else offsets
        self.mask = rng.random(tokens) < 0.7 if mask else np.ones(tokens, bool)
        self.dev_chosen = torch.from_numpy(self.chosen.astype(np.int32 if bits == 32 else np.int64)).cuda()
        self.dev_offsets = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
        self.dev_mask = torch.from_numpy(self.mask).cuda() if mask else None
        self.before = rng.standard_normal((tokens, experts + gap)).astype(np.float32)
        self.dfull = torch.from_numpy(self.before).to(kind).cuda()
        self.before = self.dfull.float().cpu().numpy()
        self.counts = torch.full((experts,), 7, dtype=torch.int64, device="cuda")
        self.loss = torch.full((1,), 5.0, device="cuda")

    def item(self, grads=True):
        e = self.experts
        return ms.router(self.full[:, :e], self.dev_chosen, self.counts, self.loss,
                         dlogits=self.dfull[:, :e] if grads else None, offsets=self.dev_offsets, mask=self.dev_mask)

    def check(self, scale=1.0, accumulate=False):
        import torch
        loss, counts, grad, bound, written = oracle(self.x, self.chosen, self.offsets, self.mask, self.score, scale)
        e = self.experts
        assert np.array_equal(self.counts.cpu().numpy(), counts + (7 if accumulate else 0))
        got = float(self.loss)
        assert abs(got - loss) <= 2.0 ** -17 * abs(loss) + 1e-30, (got, loss)
        g = self.dfull.float().cpu().numpy()
        assert np.array_equal(g[:, e:], self.before[:, e:]), "what lies between the rows"
        assert np.array_equal(g[~written], self.before[~written]), "rows of no sequence"
        half = 2.0 ** -8 if self.full.dtype == torch.bfloat16 else 2.0 ** -24
        off = np.abs(g[:, :e] - grad)[written]
        allowed = (2.0 ** -16 * bound + half * np.abs(grad))[written] + 1e-38
        assert (off <= allowed).all(), float((off / allowed).max())
        return float((off / allowed).max()) if off.size else 0.0


def run(ctx, batches, score="softmax", **kw):
    import torch
    grads = kw.pop("grads", True)
    stream = kw.pop("stream", None)
    code = ms.MUON_SCORE_SIGMOID if score == "sigmoid" else ms.MUON_SCORE_SOFTMAX
    ctx.muon_router_balance([b.item(grads) for b in batches], ms.balance_hparams(COEF, score=code, **kw), stream=stream)
    torch.cuda.synchronize()


EXPERTS = [1, 2, 7, 8, 9, 16, 17, 60, 64, 65, 128, 200, 256, 257, 384, 512, 513, 1000, 1024]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("experts", EXPERTS)
def test_expert_numbers(ctx, experts, dtype, score):
    rng = np.random.default_rng(experts)
    for tokens in (1, 3, 130):
        b = Batch(rng, tokens, experts, min(experts, 6), score=score, dtype=dtype)
        run(ctx, [b], score)
        worst = b.check()
    say(experts, dtype, score, "%.2f of the bound" % worst)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("offsets", [[0, 100, 100, 350, 351, 700], [10, 20, 20, 20, 640], [0, 0, 0], [700, 700],
                                     [5, 6], list(range(0, 701, 5))])
def test_packed_sequences(ctx, offsets, score):
    rng = np.random.default_rng(len(offsets))
    b = Batch(rng, 700, 24, 4, offsets=offsets, score=score, mask=True, gap=3, drop=0.1, bits=32)
    run(ctx, [b], score)
    b.check()


def test_many_short_sequences(ctx):
    """More sequences than a workgroup's own counts hold."""
    rng = np.random.default_rng(3)
    lengths = rng.integers(0, 4, 3000)
    offsets = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    b = Batch(rng, offsets[-1], 300, 3, offsets=offsets, dtype="f32")
    run(ctx, [b])
    b.check()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("experts", [8, 64, 100, 256])
def test_long_batches(ctx, experts, dtype, score):
    """Past what one workgroup takes: counted, balanced and finished by many; uneven sequences, mask, rows with gaps."""
    rng = np.random.default_rng(experts + 1)
    tokens = 20011
    offsets = [3, 9, 9, 5000, 5001, 12345, 20000]
    b = Batch(rng, tokens, experts, 6, offsets=offsets, score=score, dtype=dtype, mask=True, gap=5, drop=0.05)
    run(ctx, [b], score)
    say(experts, dtype, score, "%.2f of the bound" % b.check())


def test_accumulate_scale_and_no_gradient(ctx):
    import torch
    rng = np.random.default_rng(21)
    for tokens in (200, 9000):
        b = Batch(rng, tokens, 48, 4)
        scale = torch.full((1,), -3.5, device="cuda")
        run(ctx, [b], accumulate=True, grad_scale=scale)
        loss, counts, grad, bound, _ = oracle(b.x, b.chosen, b.offsets, b.mask, "softmax", -3.5)
        assert np.array_equal(b.counts.cpu().numpy(), counts + 7)
        assert (np.abs(b.dfull.cpu().numpy() - grad) <= 2.0 ** -16 * np.abs(bound) + 2.0 ** -24 * np.abs(grad)).all()
        run(ctx, [b], accumulate=True, grad_scale=scale)
        assert np.array_equal(b.counts.cpu().numpy(), 2 * counts + 7)
        kept = b.dfull.clone()
        b.loss.zero_()
        run(ctx, [b], grads=False)
        assert torch.equal(kept, b.dfull) and abs(float(b.loss) - loss) <= 2.0 ** -17 * loss
        assert np.array_equal(b.counts.cpu().numpy(), counts)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens", [64, 9000])
def test_infinities_and_vanishing_rows(ctx, tokens, score):
    """Experts that cannot be reached (-infinity, the type's lowest value), rows of nothing else, rows whose sigmoids vanish,
    large logits; masked rows hold NaN and infinities."""
    import torch
    rng = np.random.default_rng(22)
    experts = 40
    x = rng.standard_normal((tokens, experts)) * 3
    x[::7, 3:20] = -np.inf
    x[1::7] = -np.inf
    x[2::7] -= 95.0
    x[3::7, 5] = 60.0
    x[4::7, :30] = np.finfo(np.float32).min
    b = Batch(rng, tokens, experts, 4, score=score, mask=True, logits=x)
    b.mask[:] = True
    b.mask[5::7] = False
    b.dev_mask.copy_(torch.from_numpy(b.mask))
    b.full[5::7] = float("nan")
    b.full[12::14] = float("inf")
    run(ctx, [b], score)
    b.x[5::7] = 0.0
    b.check()
    assert bool((b.dfull[5::7] == 0).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens", [64, 9000])
def test_nan_rows(ctx, tokens, score):
    """A NaN logit makes its row of the gradient and the loss NaN, no other row and no count."""
    rng = np.random.default_rng(23)
    b, ref = (Batch(np.random.default_rng(23), tokens, 32, 3, score=score) for _ in range(2))
    del rng
    b.full[11, 4] = float("nan")
    run(ctx, [b, ref], score)
    assert np.isnan(float(b.loss)) and not np.isnan(float(ref.loss))
    got, want = b.dfull.cpu().numpy(), ref.dfull.cpu().numpy()
    assert np.isnan(got[11]).all()
    got[11] = want[11]
    assert np.array_equal(got, want) and np.array_equal(b.counts.cpu().numpy(), ref.counts.cpu().numpy())


def test_gradient_against_differences(ctx):
    """Central differences of the loss itself: exact loss in 64 bits at x +- h, h^2 / 6 of its third derivative below
    2^-14 of the gradient's terms for h = 2^-7."""
    rng = np.random.default_rng(24)
    for score in ("softmax", "sigmoid"):
        b = Batch(rng, 12, 10, 3, offsets=[0, 5, 12], score=score)
        run(ctx, [b], score)
        grad, h = b.dfull.cpu().numpy(), 2.0 ** -7
        bound = oracle(b.x, b.chosen, b.offsets, b.mask, score)[3]
        for t, i in [(0, 0), (3, 7), (5, 2), (11, 9)]:
            loss = []
            for sign in (1, -1):
                x = b.x.astype(np.float64)
                x[t, i] += sign * h
                loss.append(oracle(x, b.chosen, b.offsets, b.mask, score)[0])
            assert abs((loss[0] - loss[1]) / (2 * h) - grad[t, i]) <= 2.0 ** -13 * bound[t, i] + 2.0 ** -16 * bound[t, i]


def test_many_routers_and_no_tokens(ctx):
    """More routers than a launch holds, of several widths, types and lengths, some without tokens; as alone."""
    import torch
    rng = np.random.default_rng(25)
    batches = []
    for k in range(75):
        tokens = [0, 40, 3000, 5000][k % 4]
        batches.append(Batch(rng, tokens, [16, 64, 33][k % 3], 4, dtype=["f32", "bf16"][k % 2]))
    run(ctx, batches)
    for b in batches:
        b.check()
        assert b.x.shape[0] or (float(b.loss) == 0 and int(b.counts.sum()) == 0)
    before = [(b.dfull.clone(), b.loss.clone()) for b in batches]
    for b in batches:
        run(ctx, [b])
    for b, (g, loss) in zip(batches, before):
        # how tokens are spread over workgroups goes by their number: the loss's sums in another order
        assert torch.equal(b.dfull, g) and abs(float(b.loss) - float(loss)) <= 2.0 ** -23 * abs(float(loss))


def test_other_stream_and_graph(ctx):
    """Captured and replayed with eager calls of other sizes in between, small and long batches."""
    import torch
    mine = ms.Context(0)
    for tokens in (100, 9000):
        rng = np.random.default_rng(26)
        b = Batch(rng, tokens, 64, 4, offsets=[0, tokens // 3, tokens], mask=True)
        long = Batch(rng, 30000, 80, 4)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        hp = ms.balance_hparams(COEF)
        with torch.cuda.stream(side):
            mine.muon_router_balance([b.item()], hp)
        side.synchronize()
        b.check()
        want = b.dfull.clone(), b.loss.clone(), b.counts.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            mine.muon_router_balance([b.item()], hp, stream=torch.cuda.current_stream())
        for turn in range(4):
            for t in (b.dfull[:, :64], b.loss, b.counts):
                t.zero_()
            if turn % 2:
                run(mine, [long])
                long.check()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip((b.dfull, b.loss, b.counts), want)), turn
    mine.close()


def test_offsets_that_are_no_offsets(ctx):
    """Past the tokens, in front of them, descending: nothing outside the buffers is touched, whatever the result."""
    import torch
    rng = np.random.default_rng(27)
    for tokens in (100, 9000):
        for offsets in ([-50, 2 ** 31 - 1], [tokens, 0], [5, 3, -7, tokens + 9], [2 ** 31 - 1, -2 ** 31]):
            b = Batch(rng, tokens, 16, 2, offsets=offsets)
            run(ctx, [b])
            assert torch.equal(b.full.cpu(), torch.from_numpy(b.x))
    b = Batch(rng, 500, 16, 2)
    run(ctx, [b])
    b.check()


@pytest.mark.parametrize("experts", [1, 3, 64, 300, 5000])
def test_bias_step(ctx, experts):
    import torch
    rng = np.random.default_rng(experts)
    items, want, biases = [], [], []
    for k in range(130 if experts == 64 else 3):
        counts = rng.integers(0, 5, experts) * 10 ** rng.integers(0, 12)
        if k % 3 == 1:
            counts[:] = 7
        bias = rng.standard_normal(experts).astype(np.float32)
        t = torch.from_numpy(bias).cuda()
        biases.append(t)
        items.append(ms.router_bias(t, torch.from_numpy(counts.astype(np.int64)).cuda()))
        sign = [(experts * int(c) > int(counts.sum())) - (experts * int(c) < int(counts.sum())) for c in counts]
        want.append(bias - np.float32(1e-3) * np.array(sign, np.float32))
    ctx.muon_router_bias_step(items, 1e-3)
    torch.cuda.synchronize()
    for t, w in zip(biases, want):
        assert np.array_equal(t.cpu().numpy(), w)


def test_capture_needs_memory_of_an_earlier_call():
    """A long batch under capture is refused before any of the list is enqueued; a short one needs no memory."""
    import torch
    rng = np.random.default_rng(43)
    mine = ms.Context(0)
    short, long = Batch(rng, 50, 8, 2), Batch(rng, 9000, 64, 4)
    hp = ms.balance_hparams(COEF)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ms.MuonError, match="router counts"):
            mine.muon_router_balance([short.item(), long.item()], hp, stream=torch.cuda.current_stream())
        mine.muon_router_balance([short.item()], hp, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert int(short.counts.sum()) == 7 * 8 and int(long.counts.sum()) == 7 * 64
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        short.check()
        run(mine, [long])
        long.check()
    mine.close()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_offsets_past_32_bits(ctx, score):
    """Rows 2^18 elements apart: the last of them lie past 2^32 bytes; as the same rows packed, bit for bit."""
    import torch
    rng = np.random.default_rng(45)
    b = Batch(rng, 5000, 40, 3, offsets=[0, 1200, 4990], score=score, mask=True)
    run(ctx, [b], score)
    b.check()
    far = [torch.empty(4999 * (1 << 18) + 40, device="cuda").as_strided((5000, 40), (1 << 18, 1)) for _ in range(2)]
    far[0].copy_(b.full)
    far[1].copy_(torch.from_numpy(b.before))
    loss, counts = torch.zeros_like(b.loss), torch.zeros_like(b.counts)
    code = ms.MUON_SCORE_SIGMOID if score == "sigmoid" else ms.MUON_SCORE_SOFTMAX
    ctx.muon_router_balance([ms.router(far[0], b.dev_chosen, counts, loss, dlogits=far[1], offsets=b.dev_offsets,
                                       mask=b.dev_mask)], ms.balance_hparams(COEF, score=code))
    torch.cuda.synchronize()
    assert torch.equal(far[1], b.dfull) and torch.equal(loss, b.loss) and torch.equal(counts, b.counts)
    del far
    torch.cuda.empty_cache()
