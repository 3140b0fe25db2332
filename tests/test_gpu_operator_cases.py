"""perf/operators.py: its plain forms, its exact values and the library's calls on the same inputs, small and ragged."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

SIZES = "3*1+2*33+1*64+2*1407+1*10001"
TYPES = [("f32", False, "f32"), ("f32", False, "bf16"), ("bf16", False, "f32"), ("bf16", False, "bf16"),
         ("bf16", True, "f32"), ("bf16", True, "bf16")]
STATE = ("param", "master", "grad", "factor", "exp_avg", "exp_avg_scale", "exp_avg_sq", "exp_avg_sq_scale")


@pytest.fixture(scope="module")
def ops():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "operators.py")
    spec = importlib.util.spec_from_file_location("operator_cases", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _run(ops, case, own):
    import torch
    ops.own = own
    s = ops.prepare(case, 5)
    before = {k: s[k].clone() for k in STATE if s.get(k) is not None}
    out = ops.run(s)
    torch.cuda.synchronize()
    ops.own = False
    return before, out


@pytest.mark.parametrize("grad", ["f32", "bf16"])
def test_norm(ops, grad):
    case = {"op": "norm", "sizes": SIZES, "grad": grad}
    _, plain = _run(ops, case, False)
    _, ours = _run(ops, case, True)
    for ref in (plain, ops.exact(case, 5)):
        # sums in fp64 of some 13 thousand squares, 2^-53 each, and one fp32 rounding of the factor
        assert abs(float(ours["norm"]) - float(ref["norm"])) <= 1e-12 * float(ref["norm"])
        assert abs(float(ours["factor"]) - float(ref["factor"])) <= 2.0 ** -23 * float(ref["factor"])


@pytest.mark.parametrize("step", [1, 1000])
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("op", ["adamw32", "adamw8"])
def test_adamw(ops, op, types, step):
    """32-bit moments and 8-bit codes and scales bit for bit; the weights within the fp32 roundings of both sides (16
    and 12 units of 2^-24 of the update, 4 and 3 of the weight) and half a bf16 step each (2^-8).  The exact values
    hold codes as the others do, but for a second moment of zero among others, which they leave at zero: the rounding
    lifts it to the smallest code."""
    import torch
    param, master, grad = types
    case = {"op": op, "sizes": SIZES, "grad": grad, "param": param, "master": master, "clip": True, "step": step}
    before, plain = _run(ops, case, False)
    _, ours = _run(ops, case, True)
    exact = ops.exact(case, 5)
    moments = [k for k in ours if k.startswith("exp_avg")]
    for k in moments:
        assert torch.equal(ours[k].view(torch.uint8), plain[k].view(torch.uint8)), k
        if op == "adamw8":
            ref, x = exact[k], ours[k].double()
            same = (x == ref) | (torch.zeros_like(ref, dtype=torch.bool) if k != "exp_avg_sq" else (ref == 0) & (x == 2.0 ** -9))
            assert bool(same.all()), k
        else:  # three roundings of terms no larger than the sum of their magnitudes, here at most some 1e-2
            assert torch.allclose(ours[k].double(), exact[k], rtol=2.0 ** -21, atol=1e-9), k
    # The exact values take the moments unrounded.  A new first moment is off by a constant, a product and the sum, each
    # at most 2^-24 of the two terms' magnitudes together (not of their sum: they may cancel), and moves the update by
    # lr / (1 - b1^t) over the denominator times that; a new second moment by 4 x 2^-24 of itself (a constant, two
    # products and the sum of positive terms), halved by the root: 2 units of the update.
    g = (before["grad"].float() * before["factor"]).double()
    m0, v0 = before["exp_avg"].double(), before["exp_avg_sq"].double()
    if op == "adamw8":
        m0, v0 = (torch.ldexp(x.view(-1, 32), before[k].long()[:, None] - 127).flatten()
                  for x, k in ((m0, "exp_avg_scale"), (v0, "exp_avg_sq_scale")))
    v_hat = (ops.BETA2 * v0 + (1 - ops.BETA2) * g * g) / (1 - ops.BETA2 ** step)
    terms = ops.BETA1 * m0.abs() + (1 - ops.BETA1) * g.abs()
    moment = 3 * 2.0 ** -24 * ops.LR / (1 - ops.BETA1 ** step) * terms / (v_hat.sqrt() + ops.EPS)
    for k in [k for k in ("param", "master") if k in before]:
        old, new = before[k].double(), exact["param"]
        update = (new - old).abs() + ops.LR * ops.DECAY * old.abs()
        bound = 28 * 2.0 ** -24 * update + 7 * 2.0 ** -24 * torch.maximum(old.abs(), new.abs())
        if k == "param" and param == "bf16":
            bound = bound + 2 * 2.0 ** -8 * new.abs()
        assert bool(((ours[k].double() - plain[k].double()).abs() <= bound).all()), k
        assert bool(((ours[k].double() - new).abs() <= bound + moment + 2 * 2.0 ** -24 * update).all()), k
