"""muon_blocks_step on views of larger buffers and in calls of other orders and memory, against the definition."""

import math

import numpy as np
import pytest

import muon_step_amd as ms
from gpu_util import rel_fro
from test_gpu_blocks import GAMMA, LR, MU, WD, Weight, exact_o, step
from test_gpu_blocks_accuracy import EVEN, SQUARE

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = ms.Context(0)
    yield c
    c.close()


def hparams():
    return ms.make_hparams(lr=LR, momentum=MU, weight_decay=WD, gamma=GAMMA)


def nesterov(g, m):
    """M and N as the step forms them, in fp32."""
    mu = np.float32(MU)
    m = (mu * m + g).astype(np.float32)
    return m, (mu * m + g).astype(np.float32)


def test_interleaved_and_fused_views_by_the_definition(ctx):
    """Two column slices of one buffer with blocks of their own: every block's momentum, and W to O's accuracy and three
    roundings of fp32."""
    import torch
    rng = np.random.default_rng(61)
    host = {k: rng.standard_normal((192, 320)).astype(np.float32) for k in ("param", "grad", "momentum")}
    dev = {k: torch.from_numpy(x).cuda() for k, x in host.items()}
    names = ("param", "grad", "momentum")
    ctx.muon_blocks_step([ms.block_matrix(*(dev[k][:, :128] for k in names), 192, 64),
                          ms.block_matrix(*(dev[k][:, 128:] for k in names), 64, 192)], hparams())
    torch.cuda.synchronize()
    m, n = nesterov(host["grad"], host["momentum"])
    assert np.array_equal(dev["momentum"].cpu().numpy(), m) and np.array_equal(dev["grad"].cpu().numpy(), host["grad"])
    got = dev["param"].cpu().numpy().astype(np.float64)
    blocks = [(slice(None), slice(0, 64)), (slice(None), slice(64, 128))] + [(slice(64 * k, 64 * k + 64), slice(128, 320)) for k in range(3)]
    for at in blocks:
        o = exact_o(n[at]) * (LR * GAMMA * math.sqrt(192))
        kept = (1 - LR * WD) * host["param"][at].astype(np.float64)
        assert rel_fro(kept - got[at], o) <= EVEN + 3 * 2.0 ** -24 * np.linalg.norm(kept) / np.linalg.norm(o)


def test_other_orders_and_memory_by_the_definition(ctx):
    """More weights than one launch holds, of three shapes: as a list, backwards, one by one and in a context with little
    memory, each time M, O and W of every weight."""
    rng = np.random.default_rng(62)
    kinds = [((2, 2), (24, 160), EVEN), ((1, 3), (200, 40), EVEN), ((3, 1), (128, 130), SQUARE), ((2, 1), (8, 300), EVEN)]
    weights = [(Weight(rng, *kinds[k % 4][:2], "f32", "bf16"), kinds[k % 4][2]) for k in range(70 * 4)]
    start = [{k: t.clone() for k, t in w.dev.items()} for w, _ in weights]
    items = [w for w, _ in weights]
    small = ms.Context(0, workspace_cap_bytes=3 << 20)
    for how in (lambda: step(ctx, items), lambda: step(ctx, items[::-1]), lambda: [step(ctx, [w]) for w in items],
                lambda: step(small, items)):
        for (w, _), s in zip(weights, start):
            for k, t in w.dev.items():
                t.copy_(s[k])
        how()
        for w, tol in weights:
            w.check(tol)
    small.close()


@pytest.mark.parametrize("cols", [8, 200])
def test_one_row_of_a_far_pitch(ctx, cols):
    """A single row's pitch says nothing, however far the next one would be."""
    import torch
    rng = np.random.default_rng(63)
    host = [rng.standard_normal((1, cols)).astype(np.float32) for _ in range(3)]
    dev = [torch.from_numpy(x).cuda() for x in host]
    far = [t.as_strided((1, cols), (pitch, 1)) for t, pitch in zip(dev, (1 << 40, 1 << 27, 0))]
    ctx.muon_blocks_step([ms.block_matrix(*far, 1, cols)], hparams())
    torch.cuda.synchronize()
    m, n = nesterov(host[1], host[2])
    assert np.array_equal(dev[2].cpu().numpy(), m)
    want = (1 - LR * WD) * host[0].astype(np.float64) - LR * GAMMA * math.sqrt(cols) * exact_o(n)
    assert np.abs(dev[0].cpu().numpy() - want).max() <= 4 * 2.0 ** -24 * np.abs(want).max() + EVEN * LR * GAMMA * np.sqrt(cols)
