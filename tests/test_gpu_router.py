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
