"""Calls of the mixed-type AdamW steps, the gradient norm and the clip factor that their documentation allows or rules
out, where one was once answered wrongly; needs no GPU."""

import numpy as np
import pytest

import muon_step_amd as ms
import oracle


@pytest.mark.parametrize("codes", ["uint8", "float8_e4m3fn"])
@pytest.mark.parametrize("scales", ["uint8", "float8_e8m0fnu"])
def test_moments_of_every_type_a_state_may_have(codes, scales):
    """A state holds its codes and exponents as bytes or as torch's types of the same bits: the values are the same."""
    import torch
    rng = np.random.default_rng(21)
    n = 7 * 32 + 3
    c = rng.integers(0, 256, n).astype(np.uint8)
    e = np.array([0, 1, 17, 118, 127, 200, 254, 255], np.uint8)
    state = (torch.from_numpy(c).view(getattr(torch, codes)), torch.from_numpy(e).view(getattr(torch, scales))) * 2
    with np.errstate(over="ignore"):
        ref = oracle.moment_values(c, e).astype(np.float32)
    for x in ms.adamw8_moments(state):
        assert x.dtype == torch.float32 and np.array_equal(x.numpy(), ref, equal_nan=True)
