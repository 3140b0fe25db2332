"""muon_router_balance where fp32's range ends, and where memory of the context is given up for more of it."""

import numpy as np
import pytest

import muon_step_amd as ms
from test_gpu_router import Batch, oracle, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = ms.Context(0)
    yield c
    c.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens", [64, 9000])
def test_unreachable_experts_get_no_gradient(ctx, tokens, score, dtype):
    """A logit of -infinity has p 0: its gradient is 0 however large grad_scale is."""
    import torch
    rng = np.random.default_rng(51)
    x = rng.standard_normal((tokens, 40)) * 3
    x[:, ::3] = -np.inf
    x[1::5] = -np.inf
    x[2::5, 1:] = -np.inf
    b = Batch(rng, tokens, 40, 4, score=score, dtype=dtype, logits=x)
    scale = torch.full((1,), 2.0 ** 80, device="cuda")
    run(ctx, [b], score, grad_scale=scale)
    g = b.dfull.float().cpu().numpy()
    assert np.isfinite(g).all() and not g[np.isneginf(x)].any()
    assert g[3::5, 1].any()
    b.check(scale=2.0 ** 80)


@pytest.mark.parametrize("experts", [3, 40, 256])
@pytest.mark.parametrize("tokens", [64, 9000])
def test_rows_of_small_sigmoids(ctx, tokens, experts):
    """From rows whose sigmoids are below fp32's last bit of 1 to ones that fp32 cannot hold: p is as exact as elsewhere.
    Scores below 2^-126 in a row whose sum is 2^-26 or more count as none: 2^-100 of p."""
    rng = np.random.default_rng(52)
    x = rng.standard_normal((tokens, experts)) * 2
    shift = rng.choice([0, -15, -17, -18.5, -40, -60, -69, -75, -80, -84, -87, -88, -95, -104, -300, -3e4], (tokens, 1))
    wide = rng.random((tokens, experts)) * np.where(rng.random((tokens, 1)) < 0.5, 40.0, 0.0)
    b = Batch(rng, tokens, experts, min(experts, 4), score="sigmoid", logits=x + shift - wide)
    run(ctx, [b], "sigmoid")
    loss, counts, grad, bound, _ = oracle(b.x, b.chosen, b.offsets, b.mask, "sigmoid")
    away = np.abs(grad).max()
    off = np.abs(b.dfull.cpu().numpy() - grad)
    assert (off <= 2.0 ** -16 * bound + 2.0 ** -24 * np.abs(grad) + 2.0 ** -100 * away + 1e-38).all()
    assert abs(float(b.loss) - loss) <= 2.0 ** -17 * loss and np.array_equal(b.counts.cpu().numpy(), counts)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts, sequences", [(64, 20000), (256, 4096), (1000, 300), (5, 30000)])
def test_thousands_of_sequences(ctx, experts, sequences, score):
    """Sequences of no token, one and some, and masked ones; another router of few in the same launch; again, and added up."""
    import torch
    rng = np.random.default_rng(53)
    cuts = np.sort(rng.integers(0, 30001, sequences - 1)).tolist()
    mine = ms.Context(0)
    many = Batch(rng, 30000, experts, 3, offsets=[0, *cuts, 30000], mask=True, bits=32, score=score)
    few = Batch(rng, 9000, experts, 3, offsets=[0, 4000, 4000, 9000], score=score)
    none = Batch(rng, 0, experts, 3, offsets=[0] * 40, score=score)
    for turn in range(3):
        run(mine, [few, many, none], score)
        for b in (many, few, none):
            b.check()
    first = [(b.counts.clone(), b.loss.clone(), b.dfull.clone()) for b in (many, few)]
    for b in (many, few, none):
        b.counts.fill_(7)
    run(mine, [few, many, none], score, accumulate=True)
    for b, (counts, loss, grad) in zip((many, few), first):
        assert torch.equal(b.counts, counts + 7) and torch.equal(b.loss, loss) and torch.equal(b.dfull, grad)
    assert bool((none.counts == 7).all())
    graph, hp = torch.cuda.CUDAGraph(), ms.balance_hparams(1e-2, score=ms.MUON_SCORE_SIGMOID if score == "sigmoid" else ms.MUON_SCORE_SOFTMAX)
    with torch.cuda.graph(graph):
        mine.muon_router_balance([few.item(), many.item(), none.item()], hp, stream=torch.cuda.current_stream())
    for turn in range(3):
        run(mine, [few], score)
        for b in (many, few):
            b.counts.zero_()
            b.loss.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for b, kept in zip((many, few), first):
            assert all(torch.equal(x, y) for x, y in zip((b.counts, b.loss, b.dfull), kept)), turn
    mine.close()
