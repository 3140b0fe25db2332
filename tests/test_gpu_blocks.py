"""muon_blocks_step against the iteration in 64 bits: shapes, types, strides, schedules, scales, empty and spoilt blocks.

Tolerances.  M is held to its bits, W to the bits that the library's own O gives.  O's relative Frobenius error: every
product's operands are pairs of truncated 16-bit parts, 2^-20 of an operand at most with the part that falls out, so a
product is off by 2^-19 of its norm, and a step of three products with coefficients that sum to about 10 in magnitude by
10 x 2^-19 = 2e-5 where nothing grows it: 2e-4 for ten steps over matrices whose singular values lie within a factor of
ten (WELL).  In the direction of a small singular value the noise of A = X X^T grows by a^2 a step until A is taken anew,
up to 2^11 before a step that reads it (b / a of it: 1.4): 2^-19 x 2^11 x 1.4 = 5.5e-3 (SPREAD)."""

import math

import numpy as np
import pytest

import muon_step_amd as ms
from gpu_util import assert_bitexact, rel_fro, say

pytestmark = pytest.mark.gpu

WELL, SPREAD = 2e-4, 5.5e-3
HYBRID = [(3.4445, -4.7750, 2.0315)] * 8 + [(2.0, -1.5, 0.5)] * 2
QUINTIC = [(3.4445, -4.7750, 2.0315)] * 5
LR, MU, WD, GAMMA = 0.02, 0.95, 0.1, 0.2


@pytest.fixture(scope="module")
def ctx():
    c = ms.Context(0)
    yield c
    c.close()


def exact_o(n, coeffs=HYBRID):
    """The iteration in 64 bits on the smaller side."""
    x = np.asarray(n, np.float64)
    flip = x.shape[0] > x.shape[1]
    x = x.T if flip else x
    largest = np.abs(x).max()
    x = x / largest
    x = x / np.linalg.norm(x)
    for a, b, c in coeffs:
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.T if flip else x


def law(rng, kind, n, m):
    if kind == "gauss":
        return rng.standard_normal((n, m))
    s = min(n, m)
    u = np.linalg.qr(rng.standard_normal((n, s)))[0]
    v = np.linalg.qr(rng.standard_normal((m, s)))[0]
    sigma = np.exp(rng.uniform(math.log(1e-4), math.log(1e-1), s))
    return (u * sigma) @ v.T + rng.standard_normal((n, m)) * 1e-5


class Weight:
    """One weight on the host and the device, its rows `gap` elements further apart than they are long."""

    def __init__(self, rng, grid, block, param, grad, kind="gauss", gap=0, scale=1.0, momentum=True):
        import torch
        self.grid, self.block, self.gap = grid, block, gap
        rows, cols = grid[0] * block[0], grid[1] * block[1]
        g, m = (np.zeros((rows, cols)) for _ in range(2))
        for a in range(grid[0]):
            for b in range(grid[1]):
                at = (slice(a * block[0], (a + 1) * block[0]), slice(b * block[1], (b + 1) * block[1]))
                g[at] = law(rng, kind, *block) * scale
                if momentum:
                    m[at] = law(rng, kind, *block) * scale
        self.dev = {}
        pitch = cols + gap
        for name, x, dtype in (("param", rng.standard_normal((rows, cols)) * 0.02, param), ("grad", g, grad),
                               ("momentum", m, "f32"), ("ns_out", np.zeros((rows, cols)), "f32")):
            full = rng.standard_normal((rows, pitch))
            full[:, :cols] = x
            t = torch.from_numpy(full.astype(np.float32)).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
            self.dev[name] = t
        self.before = {k: t.float().cpu().numpy() for k, t in self.dev.items()}
        self.shape = (rows, cols)

    def view(self, name):
        return self.dev[name][:, :self.shape[1]]

    def item(self):
        return ms.block_matrix(self.view("param"), self.view("grad"), self.view("momentum"), *self.block, ns_out=self.view("ns_out"))

    def got(self, name):
        return self.dev[name].float().cpu().numpy()

    def check(self, tol, coeffs=HYBRID, nesterov=True, factor=None, unit_rms=False, hp=(LR, MU, WD, GAMMA), skip=()):
        """Everything against the definition; returns the largest error of a block's O."""
        import oracle
        lr, mu, wd, gamma = hp
        cols = self.shape[1]
        g = self.before["grad"][:, :cols]
        if factor is not None:
            g = (g * np.float32(factor)).astype(np.float32)
        mu32 = np.float32(mu)
        m = (mu32 * self.before["momentum"][:, :cols] + g).astype(np.float32)
        n = (mu32 * m + g).astype(np.float32) if nesterov else m
        assert_bitexact(self.got("momentum")[:, :cols], m, "momentum")
        worst = 0.0
        for name in ("param", "momentum", "grad", "ns_out"):  # what lies between the rows is as it was
            assert_bitexact(self.got(name)[:, cols:], self.before[name][:, cols:], f"{name} between the rows")
        assert_bitexact(self.got("grad"), self.before["grad"], "grad")
        o, w = self.got("ns_out"), self.got("param")
        bf16 = self.dev["param"].element_size() == 2
        for a in range(self.grid[0]):
            for b in range(self.grid[1]):
                if (a, b) in skip:
                    continue
                at = (slice(a * self.block[0], (a + 1) * self.block[0]), slice(b * self.block[1], (b + 1) * self.block[1]))
                err = rel_fro(o[at], exact_o(n[at], coeffs))
                assert err <= tol, f"block {a, b}: O rel err {err:.3e} > {tol:.1e}"
                worst = max(worst, err)
                if not unit_rms:
                    ref = oracle.apply_update_f32(self.before["param"][at], o[at], lr, wd, gamma, bf16)
                    assert_bitexact(w[at], ref, f"param of block {a, b}")
                else:
                    s = lr * gamma * math.sqrt(self.block[0] * self.block[1]) / np.linalg.norm(o[at].astype(np.float64))
                    ref = (1 - lr * wd) * self.before["param"][at].astype(np.float64) - s * o[at]
                    # ||O|| from the s x s side: the products' 2^-19, and the roundings of W
                    bound = 2.0 ** -18 * np.abs(s * o[at]) + 3 * 2.0 ** -24 * np.abs(ref) + 2.0 ** -24 * np.abs(s * o[at])
                    if bf16:
                        bound = bound + 2.0 ** -8 * np.abs(ref)
                    assert (np.abs(w[at] - ref) <= bound).all(), f"param of block {a, b}"
        return worst


def step(ctx, weights, **kw):
    import torch
    stream = kw.pop("stream", None)
    hp = ms.make_hparams(lr=LR, momentum=MU, weight_decay=WD, gamma=GAMMA, **kw)
    ctx.muon_blocks_step([w.item() for w in weights], hp, stream=stream)
    torch.cuda.synchronize()


SIDES = [1, 2, 7, 16, 31, 32, 33, 48, 64, 80, 96, 100, 127, 128]


@pytest.mark.parametrize("columns", [False, True])
@pytest.mark.parametrize("s", SIDES)
def test_sides(ctx, s, columns):
    rng = np.random.default_rng(s)
    worst = 0.0
    for l in (max(s, 2), 2 * s + 1, 257, 500):
        block, grid = ((l, s), (1, 3)) if columns else ((s, l), (3, 1))
        if l < s:
            continue
        w = Weight(rng, grid, block, "bf16", "bf16")
        step(ctx, [w])
        worst = max(worst, w.check(SPREAD if l <= 2 * s + 1 else WELL))
    say(f"s={s} columns={columns}: {worst:.2e}")


@pytest.mark.parametrize("columns", [False, True])
@pytest.mark.parametrize("param", ["f32", "bf16"])
@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("gap", [0, 1, 8])
def test_types_and_strides(ctx, param, grad, gap, columns):
    rng = np.random.default_rng(gap)
    for s, l in ((64, 515), (90, 333), (128, 1024)):
        block, grid = ((l, s), (2, 2)) if columns else ((s, l), (2, 2))
        w = Weight(rng, grid, block, param, grad, gap=gap)
        step(ctx, [w])
        w.check(WELL)


@pytest.mark.parametrize("s,l", [(16, 2048), (64, 1000), (96, 1536), (128, 2048), (128, 128)])
def test_spread_spectra(ctx, s, l):
    rng = np.random.default_rng(5)
    weights = [Weight(rng, (2, 1), (s, l), "bf16", "bf16", "spread"), Weight(rng, (1, 2), (l, s), "f32", "bf16", "spread")]
    step(ctx, weights)
    say(s, l, ["%.2e" % w.check(SPREAD) for w in weights])
