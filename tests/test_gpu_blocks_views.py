"""muon_blocks_step on views of larger buffers, against the definition."""

import math

import numpy as np
import pytest

import muon_step_amd as ms
from test_gpu_blocks import GAMMA, LR, MU, WD, exact_o
from test_gpu_blocks_accuracy import EVEN

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
