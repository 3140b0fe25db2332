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


@pytest.mark.parametrize("columns", [False, True])
def test_schedules_and_modes(ctx, columns):
    """Schedules of none, one and more steps than a segment; plain momentum; updates scaled by their own RMS; a factor."""
    import torch
    rng = np.random.default_rng(7)
    block, grid = ((700, 72), (1, 2)) if columns else ((72, 700), (2, 1))
    for coeffs in ([], [(1.5, -0.5, 0.0)], [(2.0, -1.5, 0.5)] * 20, QUINTIC, [(3.4445, -4.7750, 2.0315)] * 12):
        for unit_rms in (False, True):
            w = Weight(rng, grid, block, "f32", "f32")
            step(ctx, [w], coeffs=coeffs, scale_mode=ms.MUON_SCALE_UNIT_RMS if unit_rms else ms.MUON_SCALE_SQRT_MAX)
            w.check(WELL, coeffs=coeffs, unit_rms=unit_rms)
    w = Weight(rng, grid, block, "bf16", "bf16")
    step(ctx, [w], nesterov=False)
    w.check(WELL, nesterov=False)
    factor = torch.full((1,), 0.37, device="cuda")
    w = Weight(rng, grid, block, "bf16", "bf16")
    step(ctx, [w], grad_factor=factor)
    w.check(WELL, factor=float(factor))


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-14, 1e12, 1e20, 1e30])
def test_scale_does_not_matter(ctx, scale):
    """From gradients whose squares vanish in fp32 to ones whose squares overflow it, whole and ragged blocks."""
    rng = np.random.default_rng(9)
    weights = [Weight(rng, (2, 1), (64, 384), "f32", "f32", scale=scale),
               Weight(rng, (1, 2), (333, 50), "f32", "f32", scale=scale)]
    step(ctx, weights)
    for w in weights:
        w.check(WELL if scale > 1e-37 else 5e-3)  # at 1e-38 N itself has as few as 18 bits left: 2^-18 x what a step grows


def test_parts_of_different_scale(ctx):
    """A block most of whose columns are so small that their squares vanish, and some zero: they add nothing that counts."""
    rng = np.random.default_rng(10)
    w = Weight(rng, (1, 1), (64, 4096), "f32", "f32")
    for name in ("grad", "momentum"):
        w.dev[name][:, 256:2048] *= 1e-30
        w.dev[name][:, 2048:] = 0
        w.before[name] = w.dev[name].cpu().numpy()
    step(ctx, [w])
    w.check(WELL)


@pytest.mark.parametrize("columns", [False, True])
def test_empty_and_spoilt_blocks(ctx, columns):
    """A block of zeros decays; one with an infinity or a NaN becomes NaN as a whole; their neighbours are as ever."""
    rng = np.random.default_rng(11)
    s, l = 48, 300
    block, grid = ((l, s), (1, 5)) if columns else ((s, l), (5, 1))
    w = Weight(rng, grid, block, "f32", "bf16")

    def at(k):
        return (slice(None), slice(k * s, (k + 1) * s)) if columns else (slice(k * s, (k + 1) * s), slice(None))

    for name in ("grad", "momentum"):
        w.dev[name][at(1)] = 0
    spot = lambda k: (7, k * s + 3) if columns else (k * s + 3, 7)  # noqa: E731
    w.dev["grad"][spot(2)] = float("inf")
    w.dev["momentum"][spot(3)] = float("nan")
    w.before = {k: t.float().cpu().numpy() for k, t in w.dev.items()}
    step(ctx, [w])
    skip = {(0, k) if columns else (k, 0) for k in (1, 2, 3)}
    with np.errstate(all="ignore"):
        w.check(WELL, skip=skip)
    import oracle
    got = w.got("param")
    assert np.isnan(got[at(2)]).all() and np.isnan(got[at(3)]).all()
    assert np.isnan(w.got("ns_out")[at(2)]).all() and np.isnan(w.got("ns_out")[at(3)]).all()
    zero = np.zeros_like(w.before["param"][at(1)])
    assert_bitexact(got[at(1)], oracle.apply_update_f32(w.before["param"][at(1)], zero, LR, WD, GAMMA, False), "decay")
    # all of N a NaN, and unit RMS of zeros
    for value, mode in ((float("nan"), ms.MUON_SCALE_SQRT_MAX), (0.0, ms.MUON_SCALE_UNIT_RMS)):
        w = Weight(rng, (1, 1), (16, 100), "f32", "f32")
        for name in ("grad", "momentum"):
            w.dev[name][:] = value
        step(ctx, [w], scale_mode=mode)
        got = w.got("param")
        assert np.isnan(got).all() if value != 0 else np.array_equal(got, np.float32(1 - LR * WD) * w.before["param"])


def test_block_does_not_depend_on_the_others(ctx):
    """70 weights in one call (more than one launch holds) of three shapes, each weight alone, in other orders, in a
    context with little memory, and again: the same bits."""
    import torch
    rng = np.random.default_rng(12)
    shapes = [((2, 2), (24, 160)), ((1, 3), (200, 40)), ((3, 1), (128, 130))]
    weights = [Weight(rng, *shapes[k % 3], "bf16", "bf16") for k in range(70 * 3)]
    start = [{k: t.clone() for k, t in w.dev.items()} for w in weights]

    def again(how):
        for w, s in zip(weights, start):
            for k, t in w.dev.items():
                t.copy_(s[k])
        how()
        torch.cuda.synchronize()
        return [{k: t.clone() for k, t in w.dev.items()} for w in weights]

    ref = again(lambda: step(ctx, weights))
    small = ms.Context(0, workspace_cap_bytes=3 << 20)
    for how in (lambda: step(ctx, weights), lambda: step(ctx, weights[::-1]), lambda: [step(ctx, [w]) for w in weights],
                lambda: step(small, weights)):
        out = again(how)
        # how long columns are split goes by the number of blocks: sums in another order, O by less than WELL
        for a, b in zip(ref, out):
            assert torch.equal(a["momentum"], b["momentum"])
            assert float((a["ns_out"] - b["ns_out"]).norm()) <= WELL * float(a["ns_out"].norm())
    same = again(lambda: step(ctx, weights))
    for a, b in zip(ref, same):
        assert all(torch.equal(a[k], b[k]) for k in a), "two calls alike"
    small.close()


def test_other_stream_and_graph(ctx):
    """On a stream of its own, and captured: replays step as eager calls do, other work in between."""
    import torch
    rng = np.random.default_rng(13)
    mine = ms.Context(0)
    a, b = (Weight(np.random.default_rng(13), (2, 2), (40, 200), "bf16", "bf16") for _ in range(2))
    hp = ms.make_hparams(lr=LR, momentum=MU, weight_decay=WD, gamma=GAMMA)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(ms.MuonError) as e, torch.cuda.graph(torch.cuda.CUDAGraph(), stream=side):
        mine.muon_blocks_step([b.item()], hp, stream=torch.cuda.current_stream())
    assert e.value.status == 2
    with torch.cuda.stream(side):
        mine.muon_blocks_step([a.item()], hp)
        mine.muon_blocks_step([b.item()], hp)
    side.synchronize()
    with torch.cuda.graph(graph, stream=side):
        mine.muon_blocks_step([b.item()], hp, stream=torch.cuda.current_stream())
    other = Weight(rng, (9, 1), (128, 3000), "f32", "f32")  # grows the context's memory: the graph keeps its own
    for turn in range(4):
        mine.muon_blocks_step([a.item()], hp)
        torch.cuda.synchronize()
        if turn == 1:
            step(mine, [other])
            other.check(WELL)
        graph.replay()
        torch.cuda.synchronize()
        for name in a.dev:
            assert torch.equal(a.dev[name], b.dev[name]), (turn, name)
    mine.close()


def test_interleaved_and_fused_views(ctx):
    """Slices of the columns of one buffer as weights of their own, and a fused weight whose slices have other blocks."""
    import torch
    rng = np.random.default_rng(14)
    base = {k: torch.from_numpy(rng.standard_normal((192, 320)).astype(np.float32)).cuda() for k in ("param", "grad", "momentum")}
    whole = {k: t.clone() for k, t in base.items()}
    hp = ms.make_hparams(lr=LR, momentum=MU, weight_decay=WD, gamma=GAMMA)

    def items(d):
        left = [d[k][:, :128] for k in ("param", "grad", "momentum")]
        right = [d[k][:, 128:] for k in ("param", "grad", "momentum")]
        return [ms.block_matrix(*left, 192, 64), ms.block_matrix(*right, 64, 192)]

    ctx.muon_blocks_step(items(base), hp)
    for it in items(whole):
        ctx.muon_blocks_step([it], hp)
    torch.cuda.synchronize()
    assert torch.equal(base["momentum"], whole["momentum"])
    n = (np.float32(MU) * base["momentum"].cpu().numpy() + base["grad"].cpu().numpy()).astype(np.float64)
    scale = LR * GAMMA
    for rows, cols in [(slice(None), slice(0, 64)), (slice(None), slice(64, 128))] + [(slice(64 * k, 64 * k + 64), slice(128, 320)) for k in range(3)]:
        o = exact_o(n[rows, cols])
        moved = (1 - LR * WD) * 0 + (whole["param"][rows, cols] - base["param"][rows, cols]).cpu().numpy()
        assert np.abs(moved).max() <= 2 * WELL * scale * math.sqrt(192) * np.abs(o).max() * 8


def test_matches_muon_step(ctx):
    """A contiguous weight that is one block: muon_step's momentum bit for bit, its update within that step's 2e-2."""
    import torch
    rng = np.random.default_rng(15)
    w = Weight(rng, (1, 1), (96, 640), "bf16", "bf16")
    p, g, m, o = (w.view(k).clone() for k in ("param", "grad", "momentum", "ns_out"))
    step(ctx, [w])
    ctx.muon_step([ms.matrix(p, g, m, o)], ms.make_hparams(lr=LR, momentum=MU, weight_decay=WD, gamma=GAMMA))
    torch.cuda.synchronize()
    assert torch.equal(m, w.view("momentum"))
    assert float((o - w.view("ns_out")).norm()) <= 2e-2 * float(o.norm())


def test_long_side_past_a_launch(ctx):
    """One block of 65537 columns, and one of as many rows: 32 parts and a last column of its own."""
    rng = np.random.default_rng(16)
    weights = [Weight(rng, (1, 1), (20, 65537), "bf16", "bf16", gap=1), Weight(rng, (1, 1), (65537, 20), "bf16", "f32", gap=3)]
    step(ctx, weights)
    for w in weights:
        w.check(WELL)


def test_memory_for_all_blocks_or_none():
    """A list of which one shape does not fit the cap, or would have to grow the memory under capture, steps nothing."""
    import torch
    rng = np.random.default_rng(41)
    fits, large = Weight(rng, (1, 1), (16, 64), "f32", "f32"), Weight(rng, (2, 1), (128, 2048), "f32", "f32")
    state = lambda: [w.dev[k].clone() for w in (fits, large) for k in ("param", "momentum")]  # noqa: E731
    before = state()
    hp = ms.make_hparams(lr=LR, momentum=MU, weight_decay=WD, gamma=GAMMA)
    capped = ms.Context(0, workspace_cap_bytes=64 << 10)
    with pytest.raises(ms.MuonError, match="workspace cap"):
        capped.muon_blocks_step([fits.item(), large.item()], hp)
    capped.close()
    fresh = ms.Context(0)
    idle = Weight(rng, (1, 1), (16, 64), "f32", "f32")
    fresh.muon_blocks_step([idle.item()], hp)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ms.MuonError, match="block workspace"):
            fresh.muon_blocks_step([fits.item(), large.item()], hp, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(state(), before))
    fresh.close()


@pytest.mark.parametrize("block", [(16, 64), (64, 16)])
def test_offsets_past_32_bits(ctx, block):
    """Rows as far apart as they may be: the last of them lie past 2^32 bytes; as the same blocks packed."""
    import torch
    rng = np.random.default_rng(44)
    pitch, shape = 1 << 26, (2 * block[0] if block[0] == 16 else block[0], block[1])
    rows = shape[0]
    host = {k: rng.standard_normal(shape).astype(np.float32) for k in ("param", "grad", "momentum")}
    outs = []
    for wide in (False, True):
        t = {}
        for k, x in host.items():
            kind = torch.float32 if k == "momentum" else torch.bfloat16
            full = torch.empty(((rows - 1) * pitch + shape[1]) if wide else x.size, dtype=kind, device="cuda")
            t[k] = full.as_strided(shape, (pitch if wide else shape[1], 1))
            t[k].copy_(torch.from_numpy(x))
        ctx.muon_blocks_step([ms.block_matrix(t["param"], t["grad"], t["momentum"], *block)],
                             ms.make_hparams(lr=LR, momentum=MU, weight_decay=WD, gamma=GAMMA))
        torch.cuda.synchronize()
        outs.append((t["param"].clone(), t["momentum"].clone()))
        del t, full
        torch.cuda.empty_cache()
    assert all(torch.equal(x, y) for x, y in zip(*outs))
