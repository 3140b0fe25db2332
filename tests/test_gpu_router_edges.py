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
