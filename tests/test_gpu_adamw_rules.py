"""The mixed-type AdamW steps, the gradient norm and the clip factor on the GPU at the ends of their ranges, against
the oracle."""

import math

import numpy as np
import pytest

from test_gpu_adamw import SEED, TYPES, Case, Guarded, _bf16, _step, ctx, ms, torch  # noqa: F401  (fixtures among them)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("step", [1, 3])
def test_adamw8_large_second_moments(ctx, torch, ms, step):
    """Second moments from 2^60 to past fp32's largest value, a power of two for each block: the weights move as the
    formula has it as long as v / (1 - b2^step) is an fp32 value, and only decay from there on."""
    exponents = np.arange(30, 65)

    def change(p, g, m, v):
        for b, k in enumerate(exponents):
            s = slice(32 * b, 32 * b + 32)
            g[s] = np.ldexp(np.where(g[s] < 0, -1.0, 1.0) * (1 + np.arange(32) / 32), int(k))
            if step != 1:
                m[s] = np.ldexp(m[s], int(k))
                v[s] = np.minimum(np.ldexp(np.float64(v[s]) * 100, 2 * int(k)), 3e38)
    rng = np.random.default_rng(51)
    cases = [Case(torch, ms, True, rng, 32 * len(exponents), t, step, change=change) for t in TYPES]
    _step(ctx, ms, cases, step)
    torch.cuda.synchronize()
    for c in cases:
        c.check(step, what="large v")


@pytest.mark.parametrize("eps", [0.0, 2.0 ** -126, 1e-20, 1e-13, 2.0 ** -39, 2.0 ** -38, 1e-11, 1e-8])
def test_adamw8_small_second_moments(ctx, torch, ms, eps):
    """Gradients from 2^-77 to 2^-10, a power of two for each block, so that second moments end among the subnormal
    values and below them, with an eps that hides them and with one that does not."""
    exponents = np.arange(-77, -9)

    def change(p, g, m, v):
        for b, k in enumerate(exponents):
            s = slice(32 * b, 32 * b + 32)
            g[s] = np.ldexp(np.where(g[s] < 0, -1.0, 1.0) * (1 + np.arange(32) / 32), int(k))
    rng = np.random.default_rng(52)
    cases = [Case(torch, ms, True, rng, 32 * len(exponents), t, 1, change=change) for t in TYPES]
    _step(ctx, ms, cases, 1, eps=eps)
    torch.cuda.synchronize()
    for c in cases:
        c.check(1, eps=eps, what=f"eps {eps}")
