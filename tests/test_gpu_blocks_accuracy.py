"""How far muon_blocks_step's O is from the iteration in 64 bits: schedules of every length that is taken, and spectra.

SHORT: blocks whose singular values lie within a factor of ten.  Every product's operands are pairs of 16-bit parts, 2^-20
of an operand at most with the part that falls out.  Where nothing grows them, errors of steps add up like independent
ones, and 3e-5 is what the header gives for any of them.  A schedule that does not settle (the quintic's singular values
keep moving between 0.68 and 1.21) passes a relative error of a singular value on by sigma f'(sigma) / f(sigma) a step;
`sensitivity` is the root mean square of what a whole schedule makes of it, and any arithmetic's error has that factor.

EVEN: the same blocks in 1e-6, which the header gives, times a margin of 4.  Both parts of a pair are rounded to nearest, 2^-24
of the operand together, and lo lo is left out, 2^-24 again: a product of two is off by 3 x 2^-24, its fp32 sums over up to 24
accumulations by about as much, and the three products of a step by 10 (the coefficients' magnitudes) x 2^-22 = 2.4e-6 at most;
they are independent, and the schedule settles what it does not move.  WIDE, SQUARE: the header's figures for spectra over three
decades, where the noise of A grows by a^2 a step in small directions; a margin of two for squares, whose smallest singular
values are a matter of luck.  DEFICIENT: P's rounding, 2^-24 of its largest entries, which are the schedule's gain where N has
no direction, meets all of N; a product has two roundings of P's and N's each: four times that.

NARROW: sides up to 16, whose sums and polynomials are fp64.  What is left is the rounding in the last product, P N: two
operands and the lo lo that is left out, 3 x 2^-24 of |P| |N|.  Largest is P's u u^T / sigma along the smallest singular value
(of N / ||N||; or the schedule's gain, where that is less), so O is off by 3 x 2^-24 / sigma at most, of a norm of sqrt(s): `last_product`.
That is what holds in short blocks, whose smallest singular values are a matter of luck (10^4 below the norm in a square of
16); where noise keeps them above 10^-3.5 and 16 rows share the error, it is 6e-6 at most by emulation."""

import numpy as np
import pytest

import muon_step_amd as ms
from gpu_util import rel_fro, say
from test_gpu_blocks import HYBRID, MU, Weight, exact_o, step

pytestmark = pytest.mark.gpu

SHORT, EVEN, WIDE, SQUARE, DEFICIENT = 3e-5, 4e-6, 3e-5, 6e-4, 4 * 2.0 ** -24 * 3.4445 ** 8 * 4
NARROW = 6e-6
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


def last_product(n, coeffs):
    sigma = np.linalg.svd(np.asarray(n, np.float64) / np.linalg.norm(n), compute_uv=False)
    gain = np.prod([abs(a) for a, _, _ in coeffs])
    return EVEN + 3 * 2.0 ** -24 * min(1 / sigma[-1], gain) / np.sqrt(len(sigma))


def errors(weight, coeffs, bound=sensitivity):
    """Relative Frobenius error of O, and the sensitivity (or another bound), of each block of a stepped weight."""
    g, m = (weight.before[k][:, :weight.shape[1]] for k in ("grad", "momentum"))
    mu = np.float32(MU)
    m = (mu * m + g).astype(np.float32)
    n, o = (mu * m + g).astype(np.float32), weight.got("ns_out")[:, :weight.shape[1]]
    r, c = weight.block
    for a in range(weight.grid[0]):
        for b in range(weight.grid[1]):
            at = (slice(a * r, (a + 1) * r), slice(b * c, (b + 1) * c))
            yield rel_fro(o[at], exact_o(n[at], coeffs)), bound(n[at], coeffs)


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


@pytest.mark.parametrize("shape", [(1, 64), (7, 300), (16, 2048), (32, 500), (33, 400), (64, 1000), (72, 700), (96, 1536), (128, 2048)])
def test_even_spectra(ctx, shape):
    for coeffs in (HYBRID, [QUINTIC] * 5, [QUINTIC] * 12, [CUBIC] * 20, [SLOW] * 10, [SLOW] * 37, []):
        rng = np.random.default_rng(len(coeffs) + 1)
        weights = [Weight(rng, (2, 1), shape, "f32", "f32"), Weight(rng, (1, 2), shape[::-1], "f32", "f32")]
        step(ctx, weights, coeffs=coeffs)
        found = [e for w in weights for e in errors(w, coeffs)]
        say(shape, len(coeffs), coeffs[:1], ["%.1e of %.1f" % f for f in found])
        assert all(err <= EVEN * k for err, k in found)


@pytest.mark.parametrize("s, l, tol", [(16, 2048, WIDE), (48, 700, WIDE), (64, 1000, WIDE), (80, 1407, WIDE), (96, 1536, WIDE),
                                       (128, 2048, WIDE), (128, 128, SQUARE), (64, 64, SQUARE)])
def test_spread_spectra(ctx, s, l, tol):
    rng = np.random.default_rng(6)
    weights = [Weight(rng, (2, 1), (s, l), "f32", "f32", "spread"), Weight(rng, (1, 2), (l, s), "bf16", "f32", "spread")]
    step(ctx, weights)
    found = [err for w in weights for err, _ in errors(w, HYBRID)]
    say(s, l, ["%.1e" % f for f in found])
    assert max(found) <= tol


@pytest.mark.parametrize("shape", [(16, 2048), (33, 400), (72, 700), (128, 2048)])
def test_spread_spectra_of_other_schedules(ctx, shape):
    """Ones that settle and ones that do not, of every length."""
    polar = [(8.2872, -23.5959, 17.3004), (4.1071, -2.9479, 0.5448), (3.9487, -2.9089, 0.5518)]
    for coeffs in LENGTHS + [polar]:
        rng = np.random.default_rng(len(coeffs))
        weights = [Weight(rng, (2, 1), shape, "f32", "f32", "spread"), Weight(rng, (1, 2), shape[::-1], "f32", "f32", "spread")]
        step(ctx, weights, coeffs=coeffs)
        found = [e for w in weights for e in errors(w, coeffs)]
        say(shape, len(coeffs), coeffs[0][0], "%.1e of %.1f" % max(found))
        assert all(err <= WIDE * k for err, k in found)


@pytest.mark.parametrize("s, l", [(8, 300), (16, 2048), (64, 1000), (128, 2048)])
def test_ranks_below_the_smaller_side(ctx, s, l):
    """A quarter of the directions, and nothing but the values' own rounding in the others."""
    import torch
    rng = np.random.default_rng(8)
    weights = [Weight(rng, (2, 1), (s, l), "f32", "f32"), Weight(rng, (1, 2), (l, s), "f32", "f32")]
    for w in weights:
        left = rng.standard_normal((w.shape[0] // w.grid[0], s // 4)), rng.standard_normal((s // 4, w.shape[1] // w.grid[1]))
        full = np.tile(left[0] @ left[1], w.grid).astype(np.float32)
        for name in ("grad", "momentum"):
            w.dev[name].copy_(torch.from_numpy(full))
            w.before[name] = full
    step(ctx, weights)
    found = [err for w in weights for err, _ in errors(w, HYBRID)]
    say(s, l, ["%.1e" % f for f in found])
    assert max(found) <= DEFICIENT


@pytest.mark.parametrize("s, l", [(16, 2048), (16, 1000), (12, 2047), (16, 16), (16, 40), (13, 31), (8, 300), (5, 5), (2, 64),
                                  (1, 1), (1, 3000)])
def test_narrow_blocks(ctx, s, l):
    """Types, strides, schedules and spectra of sides up to 16, their parts and strips of all lengths."""
    for k, coeffs in enumerate((HYBRID, [QUINTIC] * 12, [CUBIC] * 22, [])):
        rng = np.random.default_rng(9 + k)
        types = [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")][k]
        for kind in ("spread", "gauss"):
            weights = [Weight(rng, (3, 2), (s, l), *types, kind, gap=k), Weight(rng, (2, 3), (l, s), *types, kind, gap=3 * k)]
            step(ctx, weights, coeffs=coeffs)
            for w in weights:
                w.check(1e-2, coeffs=coeffs)  # M and W to their bits, and what is not written
                found, cond = list(errors(w, coeffs, last_product)), [c for _, c in errors(w, coeffs)]
                say(s, l, kind, len(coeffs), "%.1e of %.1e" % max(found, key=lambda f: f[0] / f[1]))
                assert all(err <= tol * c for (err, tol), c in zip(found, cond))
                if l >= 1000 and s >= 12:
                    assert all(err <= NARROW * c for (err, _), c in zip(found, cond))
