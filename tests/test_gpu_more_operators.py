"""perf/more_operators.py: its plain forms, its exact values and the library's calls on the same inputs, small and ragged; and
the operators in one training step, as they follow each other."""

import importlib.util
import os

import numpy as np
import pytest

import muon_step_amd as ms

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "more_operators.py")
    spec = importlib.util.spec_from_file_location("more_operator_cases", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def sides(ops, case):
    import torch
    out = []
    for own in (False, True):
        ops.own = own
        s = ops.prepare(case, 5)
        out.append(ops.run(s))
        torch.cuda.synchronize()
    ops.own = False
    return (*out, ops.exact(case, 5))


@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("columns", [False, True])
@pytest.mark.parametrize("small, large", [(1, 64), (16, 100), (33, 70), (80, 1407), (128, 300)])
def test_blocks(ops, small, large, columns, nesterov):
    """The momentum within three roundings of its terms' magnitudes; the update, of the weights' difference, within 2e-3
    of its norm (a tenth of a bf16 product's) in the exact values' fp32 weights."""
    case = ops._blocks(None, 2, 3, small, large, columns, "f32", "f32", 5, True, False, nesterov)
    plain, ours, exact = sides(ops, case)
    before = ops.prepare(case, 5)
    cols = ops._weight_shape(case)[1]
    for ref in (plain, exact):
        m, r = ours["momentum"][..., :cols].double(), ref["momentum"][..., :cols].double()
        assert float((m - r).abs().max()) <= 2.0 ** -21 * float(r.abs().max())
        p, r, old = (x["param"][..., :cols].double() for x in (ours, ref, before))
        assert float((p - r).norm()) <= 2e-3 * float((r - old).norm())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("routers, tokens, experts, top, sequences, mask", [
    (1, 1, 2, 1, 1, False), (3, 700, 40, 4, 9, True), (2, 9001, 24, 6, 5, False), (1, 5000, 511, 9, 33, True)])
def test_balance(ops, routers, tokens, experts, top, sequences, mask, dtype, score):
    """Counts are equal; the loss within 2^-16; gradients within 2^-14 of the largest (rows differ in what they cancel)
    and half a step of their type on either side."""
    import torch
    plain, ours, exact = sides(ops, ops._balance(None, routers, tokens, experts, top, sequences, dtype, score, mask))
    step = 2.0 ** -7 if dtype == "bf16" else 2.0 ** -23
    for ref in (plain, exact):
        assert torch.equal(ours["counts"], ref["counts"])
        assert bool(((ours["loss"].double() - ref["loss"].double()).abs() <= 2.0 ** -16 * ref["loss"].double()).all())
        g, r = ours["dlogits"].double(), ref["dlogits"].double()
        assert bool(((g - r).abs() <= 2.0 ** -14 * r.abs().max() + step * r.abs()).all())


@pytest.mark.parametrize("routers, experts", [(1, 2), (64, 511)])
def test_bias(ops, routers, experts):
    plain, ours, exact = sides(ops, {"op": "bias", "routers": routers, "experts": experts})
    for ref in (plain, exact):  # one rounding of a sum
        assert float((ours.double() - ref.double()).abs().max()) <= 2.0 ** -24


def test_a_training_step():
    """One layer's optimizer step: the balance loss's gradient through the router's weight, the norm of all gradients, the
    clip factor in the heads' step, the experts' and the router's, then the selection biases; on one stream without a
    pause, three times, against the same in 64 bits.  The momentum and the fp32 update of one matrix carry the factor's
    rounding and the products' (the block step's 2e-4, the whole matrices' 2e-2, of the update's norm)."""
    import torch

    import oracle
    from gpu_util import BF16_TOL
    rng = np.random.default_rng(31)
    ctx = ms.Context(0)
    tokens, hidden, experts, top, heads, side = 1500, 96, 16, 3, 4, 24
    dev = lambda a, t=torch.float32: torch.from_numpy(np.ascontiguousarray(a)).to(t).cuda()  # noqa: E731
    x = dev(rng.standard_normal((tokens, hidden)))
    router_w, query, expert = (dev(rng.standard_normal(s) * 0.05) for s in ((experts, hidden), (heads * side, hidden), (64, hidden)))
    weights = {"router": router_w, "query": query, "expert": expert}
    grads = {k: torch.zeros_like(w) for k, w in weights.items()}
    fixed = {k: dev(rng.standard_normal(tuple(w.shape)) * 0.1) for k, w in weights.items()}
    moms = {k: torch.zeros_like(w) for k, w in weights.items()}
    sq = torch.zeros_like(router_w)
    bias, counts = torch.zeros(experts, device="cuda"), torch.zeros(experts, dtype=torch.int64, device="cuda")
    moved = torch.zeros(experts, dtype=torch.float64, device="cuda")
    loss, dlogits = torch.zeros(1, device="cuda"), torch.zeros(tokens, experts, device="cuda")
    norm, factor = torch.zeros(1, dtype=torch.float64, device="cuda"), torch.ones(1, device="cuda")
    offsets = torch.tensor([0, 400, 400, 1500], dtype=torch.int32, device="cuda")
    hp = ms.make_hparams(lr=0.02, momentum=0.95, weight_decay=0.1, gamma=0.2, grad_factor=factor)
    coef, scale = 0.5, torch.full((1,), 2.0, device="cuda")
    ref = {k: (w.double().cpu().numpy(), np.zeros(tuple(w.shape))) for k, w in weights.items() if k != "router"}
    for step in range(1, 4):
        logits = (x @ router_w.t()).contiguous()
        chosen = torch.topk(logits + bias, top, dim=1).indices.contiguous()
        ctx.muon_router_balance([ms.router(logits, chosen, counts, loss, dlogits=dlogits, offsets=offsets)],
                                ms.balance_hparams(coef, grad_scale=scale))
        for k in grads:
            grads[k].copy_(fixed[k] * step)
        grads["router"] += dlogits.t() @ x
        ctx.muon_grad_norm([ms.grad(g) for g in grads.values()], 1.0, norm, factor)
        ctx.muon_blocks_step([ms.block_matrix(query, grads["query"], moms["query"], side, hidden)], hp)
        ctx.muon_step([ms.matrix(expert, grads["expert"], moms["expert"])], hp)
        ctx.muon_adamw_mixed_step([ms.adamw_mixed_tensor(router_w, grads["router"], moms["router"], sq)],
                                  ms.adamw_hparams(lr=1e-3, step=step), grad_factor=factor)
        ctx.muon_router_bias_step([ms.router_bias(bias, counts)], 1e-3)
        torch.cuda.synchronize()
        host = {k: g.double().cpu().numpy() for k, g in grads.items()}
        total = np.sqrt(sum((g ** 2).sum() for g in host.values()))
        assert abs(float(norm) - total) <= 1e-12 * total
        f = min(1.0, 1.0 / total)
        assert abs(float(factor) - f) <= 2.0 ** -20
        want = torch.bincount(chosen.flatten(), minlength=experts)
        assert torch.equal(counts, want)
        moved -= 1e-3 * torch.sign(experts * want - want.sum()).double()
        assert float((bias - moved).abs().max()) <= 3 * 2.0 ** -33  # roundings of sums below 2^-8, and of the rate
        z = logits.double().requires_grad_()
        p, total_loss, c = torch.softmax(z, 1), 0.0, chosen.cpu()
        for a, b in ((0, 400), (400, 1500)):
            load = torch.bincount(c[a:b].flatten(), minlength=experts).double().cuda() * experts / (top * (b - a))
            total_loss = total_loss + coef / 2 * (load * p[a:b].mean(0)).sum()
        total_loss.backward()
        assert abs(float(loss) - total_loss.item()) <= 2.0 ** -17 * total_loss.item()
        assert float((dlogits - 2 * z.grad).abs().max()) <= 2.0 ** -14 * float(z.grad.abs().max())
        for k, blocks, tol in (("query", heads, 2e-4), ("expert", 1, BF16_TOL)):
            w, m = ref[k]
            m = 0.95 * m + f * host[k]
            n = 0.95 * m + f * host[k]
            out = np.concatenate([oracle.newton_schulz(b) for b in np.split(n, blocks)])
            rows = w.shape[0] // blocks
            new = w * (1 - 0.02 * 0.1) - 0.02 * 0.2 * np.sqrt(max(rows, w.shape[1])) * out
            got = weights[k].double().cpu().numpy()
            assert np.linalg.norm(got - new) <= (tol + 1e-5) * np.linalg.norm(new - w), k
            ref[k] = got, moms[k].double().cpu().numpy()
            assert np.linalg.norm(ref[k][1] - m) <= 1e-6 * np.linalg.norm(m), k
    ctx.close()
