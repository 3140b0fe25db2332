"""The mixed-type AdamW steps, the gradient norm and the clip factor on the GPU at the ends of their ranges, against
the oracle."""

import math

import numpy as np
import pytest

from test_gpu_adamw import SEED, TYPES, Case, Guarded, _bf16, _step, ctx, ms, torch  # noqa: F401  (fixtures among them)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("step", [1, 3])
def test_adamw8_large_second_moments(ctx, torch, ms, step):
    """Second moments from 2^60 to past fp32's largest value, a power of two for each block: the weights move as the
    formula has it as long as v / (1 - b2^step) is an fp32 value, and only decay from there on."""
    exponents = np.arange(30, 65)

    def change(p, g, m, v):
        for b, k in enumerate(exponents):
            s = slice(32 * b, 32 * b + 32)
            g[s] = np.ldexp(np.where(g[s] < 0, -1.0, 1.0) * (1 + np.arange(32) / 32), int(k))
            if step != 1:
                m[s] = np.ldexp(m[s], int(k))
                v[s] = np.minimum(np.ldexp(np.float64(v[s]) * 100, 2 * int(k)), 3e38)
    rng = np.random.default_rng(51)
    cases = [Case(torch, ms, True, rng, 32 * len(exponents), t, step, change=change) for t in TYPES]
    _step(ctx, ms, cases, step)
    torch.cuda.synchronize()
    for c in cases:
        c.check(step, what="large v")


@pytest.mark.parametrize("eps", [0.0, 2.0 ** -126, 1e-20, 1e-13, 2.0 ** -39, 2.0 ** -38, 1e-11, 1e-8])
def test_adamw8_small_second_moments(ctx, torch, ms, eps):
    """Gradients from 2^-77 to 2^-10, a power of two for each block, so that second moments end among the subnormal
    values and below them, with an eps that hides them and with one that does not."""
    exponents = np.arange(-77, -9)

    def change(p, g, m, v):
        for b, k in enumerate(exponents):
            s = slice(32 * b, 32 * b + 32)
            g[s] = np.ldexp(np.where(g[s] < 0, -1.0, 1.0) * (1 + np.arange(32) / 32), int(k))
    rng = np.random.default_rng(52)
    cases = [Case(torch, ms, True, rng, 32 * len(exponents), t, 1, change=change) for t in TYPES]
    _step(ctx, ms, cases, 1, eps=eps)
    torch.cuda.synchronize()
    for c in cases:
        c.check(1, eps=eps, what=f"eps {eps}")


SIZES = (1, 31, 32, 33, 64, 100, 255, 256, 1000, 1025, 4099)


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("eight", [False, True])
def test_nan_factor_adamw(ctx, torch, ms, eight, shift):
    """The factor of a norm that is not finite leaves NaN in every weight and moment, partial blocks and gradients of
    zero among them, and touches nothing else."""
    rng = np.random.default_rng(53)

    def change(p, g, m, v):
        g[::3] = 0
    cases = [Case(torch, ms, eight, rng, n, t, 5, shift, change) for n in SIZES for t in TYPES]
    _step(ctx, ms, cases, 5, torch.full((1,), math.nan, device="cuda"))
    torch.cuda.synchronize()
    for c in cases:
        what = f"n={c.n} {c.pd} {c.master}"
        for x in c.all:
            x.check(what)
        assert np.array_equal(c.dg.np(), c.g), what
        for x in (c.dp, c.dm) if c.master else (c.dp,):
            assert np.isnan(x.np()).all(), what
        for d, scale in zip(c.ds, (False, True, False, True)):
            if not eight:
                assert np.isnan(d.np()).all(), what
            elif scale:
                assert (d.np() == 255).all(), what
            else:
                assert (d.np() & 0x7F == 0x7F).all(), what


@pytest.mark.parametrize("scale_mode", ["sqrt_max", "unit_rms"])
@pytest.mark.parametrize("precision", ["bf16", "f32"])
@pytest.mark.parametrize("entry", ["muon_step", "muon_step_noalloc"])
def test_nan_factor_muon(ctx, torch, ms, entry, precision, scale_mode):
    """The same of a Muon step, shapes that pad among them; the context's next step is not affected."""
    rng = np.random.default_rng(54)
    shapes = [(64, 128), (128, 64), (33, 65), (65, 33), (200, 300), (256, 256), (8, 40), (1, 5)]
    kw = {"ns_precision": ms.MUON_NS_BF16 if precision == "bf16" else ms.MUON_NS_F32,
          "scale_mode": ms.MUON_SCALE_UNIT_RMS if scale_mode == "unit_rms" else ms.MUON_SCALE_SQRT_MAX}

    def new():
        out = []
        for k, (rows, cols) in enumerate(shapes):
            g = rng.standard_normal((rows, cols)).astype(np.float32)
            g[rows // 2] = 0
            host = ((rng.standard_normal((rows, cols)) * 0.02).astype(np.float32), g,
                    rng.standard_normal((rows, cols)).astype(np.float32))
            types = (torch.bfloat16 if k % 2 else torch.float32, torch.bfloat16 if k % 3 else torch.float32, torch.float32)
            out.append([Guarded(torch, _bf16(x).ravel(), d) for x, d in zip(host, types)])
        return out

    def step(tensors, factor):
        mats = [ms.matrix(*(x.t.view(s) for x in ts)) for ts, s in zip(tensors, shapes)]
        getattr(ctx, entry)(mats, ms.make_hparams(grad_factor=factor, **kw))

    bad, good, again = new(), new(), []
    for ts in good:
        again.append([Guarded(torch, x.np(), x.t.dtype) for x in ts])
    step(good, None)
    step(bad, torch.full((1,), math.nan, device="cuda"))
    step(again, None)
    torch.cuda.synchronize()
    for ts, s in zip(bad, shapes):
        for x, name in zip(ts, ("param", "grad", "momentum")):
            x.check(f"{s} {name}")
            assert np.isnan(x.np()).all() == (name != "grad"), f"{s} {name}"
    for a, b in zip(good, again):
        for x, y in zip(a, b):
            assert np.array_equal(x.np(), y.np())


def test_nan_factor_comes_from_the_norm(ctx, torch, ms):
    """An infinity in one gradient of one tensor: the norm's factor, read on the device, leaves NaN in all of them."""
    rng = np.random.default_rng(55)
    cases = [Case(torch, ms, eight, rng, n, t, 2) for eight in (False, True) for n in (33, 300) for t in TYPES]
    cases[3].dg.t[7] = -math.inf
    norm, factor = torch.zeros(1, dtype=torch.float64, device="cuda"), torch.ones(1, device="cuda")
    ctx.muon_grad_norm([ms.grad(c.dg.t) for c in cases], 1.0, norm, factor)
    for eight in (False, True):
        _step(ctx, ms, [c for c in cases if c.eight == eight], 2, factor)
    torch.cuda.synchronize()
    assert float(norm) == math.inf and math.isnan(float(factor))
    for c in cases:
        assert np.isnan(c.dp.np()).all()


def test_training_steps_captured_one_by_one(torch, ms):
    """The steps' scalars are the capture's, so a loop that replays graphs captures each step number anew: the same
    bits as eager calls, in fresh and in kept graphs, with eager work of another context between."""
    from test_gpu_adamw import _model
    captured, eager, between = ms.Context(0), ms.Context(0), ms.Context(0)
    try:
        a, b, other = (_model(torch, ms, seed) for seed in (61, 61, 62))

        def run(c, t, step):
            hp = ms.adamw_hparams(step=step)
            c.muon_grad_norm(t["grads"], 1.0, t["norm"], t["factor"])
            c.muon_adamw_mixed_step(t["mixed"], hp, grad_factor=t["factor"])
            c.muon_adamw8_step(t["eight"], hp, seed=SEED, grad_factor=t["factor"])

        graphs = []
        for step in range(1, 5):
            torch.cuda.synchronize()
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                run(captured, a, step)
        for step, graph in enumerate(graphs, 1):
            for x, y in zip(a["g"], b["g"]):
                x.mul_(1.0 - 0.1 * step)
                y.copy_(x)
            graph.replay()
            run(between, other, step)
            run(eager, b, step)
            torch.cuda.synchronize()
            for x, y in zip(a["state"], b["state"]):
                assert bool((x.view(torch.uint8) == y.view(torch.uint8)).all()), f"step {step}"
    finally:
        torch.cuda.synchronize()
        for c in (captured, eager, between):
            c.close()


def test_clipped_noalloc_steps_captured(torch, ms):
    """The norm and two muon_step_noalloc calls that read its factor in one graph, more matrices than one descriptor
    launch carries among them.  Between the replays the same context steps other, smaller matrices eagerly: a replay
    goes on with its own, bit for bit as eager calls do."""
    rng = np.random.default_rng(63)

    def matrices(shapes):
        return [[torch.from_numpy(rng.standard_normal(s).astype(np.float32) * k).cuda().to(d)
                 for k, d in ((0.02, torch.bfloat16), (1, torch.bfloat16), (1, torch.float32))] for s in shapes]

    def copy(ts):
        return [[x.clone() for x in t] for t in ts]

    def run(c, t):
        c.muon_grad_norm([ms.grad(g) for part in t["parts"] for _, g, _ in part], 1.0, t["norm"], t["factor"])
        for part in t["parts"]:
            c.muon_step_noalloc([ms.matrix(*x) for x in part], ms.make_hparams(grad_factor=t["factor"]))

    def state(t):
        return [x for part in t["parts"] for w, _, m in part for x in (w, m)]

    a = {"parts": [matrices([(64, 128)] * 100 + [(128, 64)] * 70), matrices([(300, 200), (5, 3)])]}
    b = {"parts": [copy(part) for part in a["parts"]]}
    for t in (a, b):
        t["norm"], t["factor"] = torch.zeros(1, dtype=torch.float64, device="cuda"), torch.zeros(1, device="cuda")
    small = matrices([(2, 2), (3, 5)])
    graph_ctx, eager_ctx = ms.Context(0), ms.Context(0)
    try:
        graph_ctx.muon_step_noalloc([ms.matrix(*x) for x in small], ms.make_hparams())
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(graph_ctx, a)
        for x, y in zip(state(a), state(b)):
            assert torch.equal(x, y), "a capture runs nothing"
        for k in range(4):
            for p, q in zip(a["parts"], b["parts"]):
                for (_, g, _), (_, h, _) in zip(p, q):
                    g.mul_(0.9)
                    h.copy_(g)
            graph_ctx.muon_step_noalloc([ms.matrix(*x) for x in small[k % 2:]], ms.make_hparams())
            graph.replay()
            run(eager_ctx, b)
            torch.cuda.synchronize()
            assert float(a["norm"]) == float(b["norm"])
            for x, y in zip(state(a), state(b)):
                assert torch.equal(x, y), f"replay {k}"
    finally:
        torch.cuda.synchronize()
        for c in (graph_ctx, eager_ctx):
            c.close()


def test_clipped_muon_and_adamw_steps_captured(torch, ms):
    """muon_step and muon_adamw_step under capture: refused on a context whose last call had another list, with the
    next eager call unharmed; otherwise the replays go on with their own tensors, whatever lists and sizes the context
    steps eagerly between them."""
    rng = np.random.default_rng(64)

    def matrices(shapes):
        return [[torch.from_numpy(rng.standard_normal(s).astype(np.float32) * k).cuda().to(d)
                 for k, d in ((0.02, torch.bfloat16), (1, torch.bfloat16), (1, torch.float32))] for s in shapes]

    def vectors(sizes):
        return [[torch.from_numpy((rng.standard_normal(n) ** 2).astype(np.float32)).cuda() for _ in range(4)] for n in sizes]

    def run(c, mats, tensors, factor):
        c.muon_step([ms.matrix(*x) for x in mats], ms.make_hparams(grad_factor=factor))
        c.muon_adamw_step([ms.adamw_tensor(*x) for x in tensors], ms.adamw_hparams(step=3))

    a = matrices([(64, 128), (128, 64), (40, 40)]), vectors([100, 7])
    b = tuple([[x.clone() for x in t] for t in part] for part in a)
    others = [(matrices(s), vectors(n)) for s, n in (([(2, 3)], [1]), ([(512, 700)] * 3 + [(64, 64)], [9, 5000, 3]))]
    factor = torch.full((1,), 0.25, device="cuda")
    graph_ctx, eager_ctx = ms.Context(0), ms.Context(0)
    try:
        for warm in (None, others[0]):
            if warm:
                run(graph_ctx, *warm, None)
            torch.cuda.synchronize()
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                for call in (lambda: graph_ctx.muon_step([ms.matrix(*x) for x in a[0]], ms.make_hparams()),
                             lambda: graph_ctx.muon_adamw_step([ms.adamw_tensor(*x) for x in a[1]], ms.adamw_hparams())):
                    with pytest.raises(ms.MuonError) as err:
                        call()
                    assert err.value.status == ms.MUON_ERR_UNSUPPORTED and "capture" in str(err.value)
                factor.add_(0)   # a graph that holds something
        run(graph_ctx, *a, factor)
        run(eager_ctx, *b, factor)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(graph_ctx, *a, factor)
        for k in range(4):
            factor.fill_(0.5 + 0.125 * k)
            run(graph_ctx, *others[k % 2], factor)
            graph.replay()
            run(eager_ctx, *b, factor)
            torch.cuda.synchronize()
            for p, q in zip(a, b):
                for t, u in zip(p, q):
                    for x, y in zip(t, u):
                        assert torch.equal(x, y), f"replay {k}"
    finally:
        torch.cuda.synchronize()
        for c in (graph_ctx, eager_ctx):
            c.close()


@pytest.mark.parametrize("count", [58, 59, 60, 64, 65, 130])
@pytest.mark.parametrize("eight", [False, True])
def test_more_tensors_of_one_kind_than_a_launch_takes(ctx, torch, ms, eight, count):
    """Around the number of tensors that one launch's arguments hold, and past two of them."""
    rng = np.random.default_rng(65)
    cases = [Case(torch, ms, eight, rng, int(rng.integers(1, 700)), ("bf16", True, "bf16"), 2) for _ in range(count)]
    _step(ctx, ms, cases, 2, torch.full((1,), 0.5, device="cuda"))
    torch.cuda.synchronize()
    for c in cases:
        c.check(2, 0.5)
