"""How far muon_blocks_step's O is from the iteration in 64 bits: schedules of every length that is taken.

SHORT: blocks whose singular values lie within a factor of ten.  Every product's operands are pairs of 16-bit parts, 2^-20
of an operand at most with the part that falls out.  Where nothing grows them, errors of steps add up like independent
ones, and 3e-5 is what the header gives for any of them.  A schedule that does not settle (the quintic's singular values
keep moving between 0.68 and 1.21) passes a relative error of a singular value on by sigma f'(sigma) / f(sigma) a step;
`sensitivity` is the root mean square of what a whole schedule makes of it, and any arithmetic's error has that factor."""

import numpy as np
import pytest

import muon_step_amd as ms
from gpu_util import rel_fro, say
from test_gpu_blocks import HYBRID, LR, MU, WD, GAMMA, Weight, exact_o, step

pytestmark = pytest.mark.gpu

SHORT = 3e-5
QUINTIC, CUBIC, SLOW = (3.4445, -4.7750, 2.0315), (2.0, -1.5, 0.5), (1.5, -0.5, 0.0)


@pytest.fixture(scope="module")
def ctx():
    c = ms.Context(0)
    yield c
    c.close()


def sensitivity(n, coeffs):
    """Root mean square over N's singular values of the schedule's relative condition number, at least 1."""
    x = np.linalg.svd(np.asarray(n, np.float64) / np.linalg.norm(n), compute_uv=False)
    k = np.ones_like(x)
    for a, b, c in coeffs:
        f = a * x + b * x ** 3 + c * x ** 5
        k, x = k * (a + 3 * b * x ** 2 + 5 * c * x ** 4) * x / f, f
    return max(1.0, float(np.sqrt((k ** 2).mean())))


def errors(weight, coeffs):
    """Relative Frobenius error of O, and the sensitivity, of each block of a stepped weight (fp32, plain layouts)."""
    g, m = (weight.before[k][:, :weight.shape[1]] for k in ("grad", "momentum"))
    mu = np.float32(MU)
    m = (mu * m + g).astype(np.float32)
    n, o = (mu * m + g).astype(np.float32), weight.got("ns_out")[:, :weight.shape[1]]
    r, c = weight.block
    for a in range(weight.grid[0]):
        for b in range(weight.grid[1]):
            at = (slice(a * r, (a + 1) * r), slice(b * c, (b + 1) * c))
            yield rel_fro(o[at], exact_o(n[at], coeffs)), sensitivity(n[at], coeffs)


# the longest of each that is taken, and shorter ones
LENGTHS = ([[QUINTIC] * n for n in (1, 2, 3, 4, 5, 8, 10, 12)] + [[CUBIC] * n for n in (1, 7, 15, 22)] +
           [[SLOW] * n for n in (2, 18, 30, 37)] + [[QUINTIC] * 8 + [CUBIC] * n for n in (1, 2, 4, 7)] + [[QUINTIC] * 10 + [CUBIC] * 4])


@pytest.mark.parametrize("shape", [(1, 64), (1, 1), (16, 2048), (33, 400), (72, 700), (128, 2048)])
def test_schedules_of_every_length(ctx, shape):
    for coeffs in LENGTHS:
        rng = np.random.default_rng(len(coeffs))
        wide, tall = Weight(rng, (2, 1), shape, "f32", "f32"), Weight(rng, (1, 2), shape[::-1], "f32", "f32")
        step(ctx, [wide, tall], coeffs=coeffs)
        for w in (wide, tall):
            for err, k in errors(w, coeffs):
                assert err <= SHORT * k, f"{len(coeffs)} steps from {coeffs[0]}: {err:.2e}, sensitivity {k:.1f}"
        say(shape, len(coeffs), coeffs[0][0], "%.1e of %.1f" % max(errors(wide, coeffs)))
