"""muon_blocks_step with sides up to 16, which have kernels of their own: scales, zeros, infinities and NaN, modes, factor,
streams, captured calls, other sides in the same call."""

import numpy as np
import pytest

import muon_step_amd as ms
from gpu_util import assert_bitexact
from test_gpu_blocks import GAMMA, LR, MU, WD, Weight, step
from test_gpu_blocks_accuracy import EVEN

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = ms.Context(0)
    yield c
    c.close()


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-14, 1e12, 1e20, 1e30, 1e37])
def test_scale_does_not_matter(ctx, scale):
    """At 1e-38 N itself has as few as 18 bits left: 2^-18 times what the steps grow."""
    rng = np.random.default_rng(71)
    weights = [Weight(rng, (2, 1), (16, 384), "f32", "f32", scale=scale), Weight(rng, (1, 2), (333, 11), "f32", "f32", scale=scale)]
    step(ctx, weights)
    for w in weights:
        w.check(EVEN if scale > 1e-37 else 5e-3)


def test_parts_of_different_scale(ctx):
    rng = np.random.default_rng(72)
    w = Weight(rng, (1, 1), (12, 4096), "f32", "f32")
    for name in ("grad", "momentum"):
        w.dev[name][:, 256:2048] *= 1e-30
        w.dev[name][:, 2048:] = 0
        w.before[name] = w.dev[name].cpu().numpy()
    step(ctx, [w])
    w.check(EVEN)


@pytest.mark.parametrize("columns", [False, True])
@pytest.mark.parametrize("s", [1, 9, 16])
def test_empty_and_spoilt_blocks(ctx, s, columns):
    """A block of zeros decays; one with an infinity or a NaN becomes NaN as a whole; their neighbours are as ever."""
    import oracle
    rng = np.random.default_rng(73)
    l = 300
    block, grid = ((l, s), (1, 6)) if columns else ((s, l), (6, 1))
    w = Weight(rng, grid, block, "f32", "bf16")
    at = lambda k: (slice(None), slice(k * s, (k + 1) * s)) if columns else (slice(k * s, (k + 1) * s), slice(None))  # noqa: E731
    spot = lambda k: (299, k * s + s // 2) if columns else (k * s + s // 2, 299)  # noqa: E731
    for name in ("grad", "momentum"):
        w.dev[name][at(1)] = 0
    w.dev["grad"][spot(2)] = float("inf")
    w.dev["momentum"][spot(3)] = float("nan")
    w.dev["momentum"][spot(5)] = float("-inf")
    w.before = {k: t.float().cpu().numpy() for k, t in w.dev.items()}
    step(ctx, [w])
    skip = {(0, k) if columns else (k, 0) for k in (1, 2, 3, 5)}
    with np.errstate(all="ignore"):
        w.check(EVEN, skip=skip)
    got = w.got("param")
    for k in (2, 3, 5):
        assert np.isnan(got[at(k)]).all() and np.isnan(w.got("ns_out")[at(k)]).all()
    zero = np.zeros_like(w.before["param"][at(1)])
    assert_bitexact(got[at(1)], oracle.apply_update_f32(w.before["param"][at(1)], zero, LR, WD, GAMMA, False), "decay")
    for value, mode in ((float("nan"), ms.MUON_SCALE_SQRT_MAX), (0.0, ms.MUON_SCALE_UNIT_RMS)):
        w = Weight(rng, (1, 1), block, "f32", "f32")
        for name in ("grad", "momentum"):
            w.dev[name][:] = value
        step(ctx, [w], scale_mode=mode)
        got = w.got("param")
        assert np.isnan(got).all() if value != 0 else np.array_equal(got, np.float32(1 - LR * WD) * w.before["param"])


@pytest.mark.parametrize("columns", [False, True])
def test_modes(ctx, columns):
    """Plain momentum, updates scaled by their own RMS with schedules of none and more steps, a factor."""
    import torch
    rng = np.random.default_rng(74)
    block, grid = ((700, 10), (1, 2)) if columns else ((10, 700), (2, 1))
    for coeffs in ([], [(1.5, -0.5, 0.0)], [(2.0, -1.5, 0.5)] * 20, [(3.4445, -4.7750, 2.0315)] * 5):
        w = Weight(rng, grid, block, "f32", "f32")
        step(ctx, [w], coeffs=coeffs, scale_mode=ms.MUON_SCALE_UNIT_RMS)
        w.check(EVEN * 3, coeffs=coeffs, unit_rms=True)  # (the quintic's sensitivity: below 3 here)
    w = Weight(rng, grid, block, "bf16", "bf16")
    step(ctx, [w], nesterov=False)
    w.check(EVEN, nesterov=False)
    for value in (0.37, 1e-20, 3e4):
        factor = torch.full((1,), value, device="cuda")
        w = Weight(rng, grid, block, "bf16", "bf16", momentum=False)
        step(ctx, [w], grad_factor=factor)
        w.check(EVEN, factor=float(factor))


def test_stream_graph_and_other_sides(ctx):
    """Sides of 16 and 17 in one call, on a stream of its own and captured: replays step as eager calls do."""
    import torch
    mine = ms.Context(0)
    make = lambda: [Weight(np.random.default_rng(75 + k), g, b, "bf16", "bf16", gap=k)  # noqa: E731
                    for k, (g, b) in enumerate((((2, 2), (16, 200)), ((3, 1), (17, 200)), ((1, 3), (500, 7))))]
    a, b = make(), make()
    hp = ms.make_hparams(lr=LR, momentum=MU, weight_decay=WD, gamma=GAMMA)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mine.muon_blocks_step([w.item() for w in a], hp)
        mine.muon_blocks_step([w.item() for w in b], hp)
    side.synchronize()
    for w in a:
        w.check(EVEN)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        mine.muon_blocks_step([w.item() for w in b], hp, stream=torch.cuda.current_stream())
    other = Weight(np.random.default_rng(79), (40, 1), (16, 9000), "f32", "f32")  # grows the context's memory
    for turn in range(4):
        mine.muon_blocks_step([w.item() for w in a], hp)
        torch.cuda.synchronize()
        if turn == 1:
            step(mine, [other])
            other.check(EVEN)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(a, b):
            for name in x.dev:
                assert torch.equal(x.dev[name], y.dev[name]), (turn, name)
    mine.close()
