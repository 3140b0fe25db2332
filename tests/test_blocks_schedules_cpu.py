"""Which schedules muon_blocks_step takes: up to a gain of 2^22 for vanishing singular values, and only those that keep the
largest singular value in reach of its fp16 pairs."""

import pytest

import muon_step_amd as ms
from test_blocks_router_cpu import block, check_blocks

QUINTIC, CUBIC, SLOW = (3.4445, -4.7750, 2.0315), (2.0, -1.5, 0.5), (1.5, -0.5, 0.0)


def taken(coeffs):
    st, msg = check_blocks([block()], ms.make_hparams(coeffs=coeffs))
    assert st in (ms.MUON_OK, ms.MUON_ERR_UNSUPPORTED) and (st == ms.MUON_OK) == (msg == ""), (st, msg)
    assert st == ms.MUON_OK or "schedule" in msg
    return st == ms.MUON_OK


@pytest.mark.parametrize("coeffs, longest", [(QUINTIC, 12), (CUBIC, 22), (SLOW, 37)])
def test_the_gain_ends_at_22_bits(coeffs, longest):
    """3.4445^12 = 2^21.4, 2^22, 1.5^37 = 2^21.6: one step more passes it, and so do many more."""
    for n in range(1, 65):
        assert taken([coeffs] * n) == (n <= longest), n


def test_mixed_schedules():
    assert taken([]) and taken([QUINTIC] * 8 + [CUBIC] * 7) and taken([QUINTIC] * 10 + [CUBIC] * 4)
    assert not taken([QUINTIC] * 8 + [CUBIC] * 8) and not taken([CUBIC] * 8 + [QUINTIC] * 8)
    assert taken(ms.schedule("deepseekv4")) and taken(ms.schedule("quintic"))


@pytest.mark.parametrize("coeffs", [
    [(0.0, 1.0, 0.0)] * 2, [(0.0, 1.0, 0.0)], [(0.0, 0.0, 1.0)], [(0.0, 0.0, 0.0)], [(0.4, 0.0, 0.0)], [(0.9, 0.0, 0.0)] * 30,
    [(0.7, 0.3, 0.0)] * 2, [(1.0, -1.0, 0.0)], [(1.0, -2.0, 0.0)], [(1.0, 0.0, -1.0)], [(1.0, 0.0, -1.1)], [(-1.0, 4.0, 0.0)], [(1e-300, 0.0, 0.0)]])
def test_schedules_that_shrink(coeffs):
    """Maps that take a singular value of [128^-1/2, 1], of which N's largest may be any, to zero or far below (0.7 x +
    0.3 x^3 twice: 0.0884 to 0.0434)."""
    assert not taken(coeffs)


@pytest.mark.parametrize("coeffs", [[(1.0, 0.0, 0.0)] * 64, [(-1.0, 0.0, 0.0)], [(-1.5, 0.5, 0.0)] * 4, [(0.6, 0.0, 0.0)],
                                    [(0.7, 0.3, 0.0)], [(8.2872, -23.5959, 17.3004), (4.1071, -2.9479, 0.5448)]])
def test_schedules_that_hold(coeffs):
    assert taken(coeffs)
