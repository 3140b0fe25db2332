"""The mixed-type AdamW steps (moments in 32 and in 8 bits), the gradient norm and the clip factor on the GPU, against
the oracle.  Every call goes through the C ABI; every tensor lies between guard elements that must stay as they are."""

import math

import numpy as np
import pytest

import oracle
from gpu_util import BF16_TOL, assert_bitexact, rel_fro, say, to_np

pytestmark = pytest.mark.gpu

LR, B1, B2, EPS, WD = 0.02, 0.9, 0.95, 1e-8, 0.1
SEED = 0x1234_5678_9ABC
GUARD = 64      # elements before and behind every tensor
SIZES = (0, 1, 7, 8, 31, 32, 33, 63, 64, 100, 255, 256, 1000, 1023, 1024, 1025, 2047, 2048, 2049, 10001, 70003)
TYPES = [("f32", False, "f32"), ("f32", False, "bf16"), ("bf16", False, "f32"), ("bf16", False, "bf16"),
         ("bf16", True, "f32"), ("bf16", True, "bf16")]


@pytest.fixture(scope="module")
def torch():
    import torch
    assert torch.cuda.is_available()
    return torch


@pytest.fixture(scope="module")
def ms():
    import muon_step_amd
    return muon_step_amd


@pytest.fixture(scope="module")
def ctx(torch, ms):
    c = ms.Context(0)
    yield c
    torch.cuda.synchronize()
    c.close()


class Guarded:
    """A device tensor of `values` between guards; `shift` elements off the allocation's alignment."""

    def __init__(self, torch, values, dtype, shift=0):
        self.torch = torch
        values = np.ascontiguousarray(values)
        src = torch.from_numpy(values)
        one = src.new_ones(1).to(dtype) if dtype != torch.uint8 else torch.full((1,), 0xA5, dtype=torch.uint8)
        self.whole = one.repeat(values.size + 2 * GUARD + shift).cuda()
        self.mark = one
        self.at = GUARD + shift
        self.t = self.whole[self.at:self.at + values.size]
        self.t.copy_(src.to(dtype))

    def check(self, what):
        behind = self.whole[self.at + self.t.numel():]
        same = bool((self.whole[:self.at].cpu() == self.mark).all()) and bool((behind.cpu() == self.mark).all())
        assert same, f"{what}: memory outside the tensor was written"

    def np(self):
        return self.t.cpu().numpy() if self.t.dtype == self.torch.uint8 else to_np(self.t)


def _bf16(x):
    return oracle.bf16_round_f32(x)


def _dtype(torch, name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _values(rng, n, step):
    p = (rng.standard_normal(n) * 0.02).astype(np.float32)
    g = (rng.standard_normal(n) * np.exp(rng.standard_normal(n))).astype(np.float32)
    m = (rng.standard_normal(n) * 0.1).astype(np.float32)
    v = (rng.standard_normal(n) ** 2 * 1e-2).astype(np.float32)
    if step == 1:
        m[:], v[:] = 0, 0
    return p, g, m, v


class Case:
    """One tensor of a step, on the host and on the device."""

    def __init__(self, torch, ms, eight, rng, n, types, step, shift=0, change=None):
        self.pd, self.master, self.gd = types
        self.n, self.eight = n, eight
        p, g, m, v = _values(rng, n, step)
        if change:
            change(p, g, m, v)
        self.p = _bf16(p) if self.pd == "bf16" and not self.master else p
        self.g = _bf16(g) if self.gd == "bf16" else g
        self.dp = Guarded(torch, p, _dtype(torch, self.pd), shift)
        self.dm = Guarded(torch, p, torch.float32, shift) if self.master else None
        self.dg = Guarded(torch, g, _dtype(torch, self.gd), shift)
        self.all = [x for x in (self.dp, self.dm, self.dg) if x]
        master = self.dm.t if self.master else None
        if eight:
            with np.errstate(invalid="ignore"):
                mc, me = oracle.quantise(m, False, np.arange(n), 1, 1, 0)
                vc, ve = oracle.quantise(v, True, np.arange(n), 1, 1, 16)
            self.state = (mc, me, vc, ve)
            self.ds = [Guarded(torch, a, torch.uint8, shift) for a in self.state]
            self.desc = ms.adamw8_tensor(self.dp.t, self.dg.t, tuple(d.t for d in self.ds), master=master)
        else:
            self.state = (m, v)
            self.ds = [Guarded(torch, a, torch.float32, shift) for a in self.state]
            self.desc = ms.adamw_mixed_tensor(self.dp.t, self.dg.t, self.ds[0].t, self.ds[1].t, master=master)
        self.all += self.ds

    def check(self, step, factor=None, seed=SEED, eps=EPS, what=""):
        what = f"{what} n={self.n} {self.pd}{'+master' if self.master else ''} grad {self.gd}"
        for x in self.all:
            x.check(what)
        assert_bitexact(self.dg.np(), self.g, what + ": the gradient is only read")
        got = self.dm.np() if self.master else self.dp.np()
        with np.errstate(all="ignore"):
            if self.eight:
                ref, update, state = oracle.adamw8_step(self.p, self.g, self.state, LR, B1, B2, eps, WD, step, seed,
                                                        factor)
            else:
                g = self.g if factor is None else np.float32(factor) * self.g
                ref, m, v = oracle.adamw_step_f32(self.p, g, *self.state, LR, B1, B2, eps, WD, step)
        if not self.eight:
            if self.pd == "bf16" and not self.master:
                ref = _bf16(ref)
            assert_bitexact(got, ref, what + ": weights")
            assert_bitexact(self.ds[0].np(), m, what + ": exp_avg")
            assert_bitexact(self.ds[1].np(), v, what + ": exp_avg_sq")
        else:
            for d, ref_bytes, name in zip(self.ds, state, ("exp_avg", "its scale", "exp_avg_sq", "its scale")):
                have = d.np()
                if name.startswith("exp"):   # the two NaN codes are one
                    have, ref_bytes = (np.where(a & 0x7F == 0x7F, 0x7F, a) for a in (have, ref_bytes))
                bad = np.flatnonzero(have != ref_bytes)
                assert bad.size == 0, f"{what}: {bad.size} of {name}'s bytes differ, first at {bad[:5]}"
            # In units of 2^-24 of the update: its constant 1 and product 1; under the root a constant 1 and a
            # product 1, halved by it; the hardware's root and reciprocal 2 each; eps and the sum with it 2: 9, and
            # 16 are allowed.  In units of 2^-24 of the larger of old and new weight: the decay's constant, its
            # product and the sum 3, and 4 are allowed.  A bf16 result is off by half a step more (2^-8 of it).
            bound = 2.0 ** -20 * np.abs(update) + 2.0 ** -22 * np.maximum(np.abs(ref), np.abs(self.p))
            if self.pd == "bf16" and not self.master:
                bound = bound + 2.0 ** -8 * np.abs(ref)
            # A reference past fp32's largest value, (2 - 2^-23) 2^127, by half a step rounds to infinity there.
            with np.errstate(invalid="ignore", over="ignore"):
                ok = (np.abs(got - ref) <= bound) | (np.isnan(got) & np.isnan(ref)) | (got == ref.astype(np.float32))
            assert ok.all(), f"{what}: weights {np.flatnonzero(~ok)[:5]}: {got[~ok][:5]} {ref[~ok][:5]}"
        if self.master:
            assert_bitexact(self.dp.np(), _bf16(self.dm.np()), what + ": the weights round the master copy")

    def raw(self):
        return [x.whole.view(self.dp.torch.uint8).cpu().clone() for x in self.all]


def _step(ctx, ms, cases, step, factor=None, seed=SEED, eps=EPS, stream=None, table=False):
    hp = ms.adamw_hparams(lr=LR, beta1=B1, beta2=B2, eps=eps, weight_decay=WD, step=step)
    descs = [c.desc for c in cases]
    if table:
        descs = ms.table(descs)
    if cases[0].eight:
        ctx.muon_adamw8_step(descs, hp, seed=seed, grad_factor=factor, stream=stream)
    else:
        ctx.muon_adamw_mixed_step(descs, hp, grad_factor=factor, stream=stream)


def _cases(torch, ms, eight, seed, step, shift=0, sizes=SIZES, types=TYPES, change=None):
    rng = np.random.default_rng(seed)
    return [Case(torch, ms, eight, rng, n, t, step, shift, change) for n in sizes for t in types]


# ------------------------------------------------------------------------------------------------------ steps

@pytest.mark.parametrize("shift", [0, 1, 3, 4, 8])
@pytest.mark.parametrize("step", [1, 7])
@pytest.mark.parametrize("eight", [False, True])
def test_step_against_oracle(ctx, torch, ms, eight, step, shift):
    """Every size and type in one call (more tensors than one launch takes, of six kinds), aligned and not."""
    cases = _cases(torch, ms, eight, 10 * step + shift, step, shift)
    clip = torch.tensor([0.37], device="cuda") if step == 7 else None
    _step(ctx, ms, cases, step, clip)
    torch.cuda.synchronize()
    for c in cases:
        c.check(step, 0.37 if clip is not None else None)
    say(f"{'8' if eight else '32'}-bit moments, step {step}, shift {shift}: {len(cases)} tensors")


@pytest.mark.parametrize("eight", [False, True])
def test_several_steps(ctx, torch, ms, eight):
    """Three steps in a row from zero moments, each checked from the state the last one left."""
    rng = np.random.default_rng(5)
    cases = [Case(torch, ms, eight, rng, n, t, 1) for n in (33, 5000) for t in TYPES]
    for step in (1, 2, 3):
        _step(ctx, ms, cases, step, table=True)
        torch.cuda.synchronize()
        for c in cases:
            c.check(step, what=f"step {step}")
            c.state = tuple(d.np().copy() for d in c.ds)
            c.p = (c.dm if c.master else c.dp).np().copy()


def test_fp32_equals_adamw_step(ctx, torch, ms):
    """fp32 tensors get the bits of muon_adamw_step."""
    rng = np.random.default_rng(6)
    hp = ms.adamw_hparams(step=3)
    for n in (1, 1000, 4099):
        host = _values(rng, n, 3)
        a, b = [[torch.from_numpy(x).cuda() for x in host] for _ in range(2)]
        ctx.muon_adamw_step([ms.adamw_tensor(*a)], hp)
        ctx.muon_adamw_mixed_step([ms.adamw_mixed_tensor(*b)], hp)
        torch.cuda.synchronize()
        for x, y in zip(a, b):
            assert_bitexact(to_np(y), to_np(x), f"n={n}")


@pytest.mark.parametrize("eight", [False, True])
def test_result_does_not_depend_on_the_call(ctx, torch, ms, eight):
    """The same tensors in one call, in another order, one by one, and from a list or a table."""
    sizes = (5, 64, 3000, 2048) * 3
    runs = []
    for how in range(4):
        cases = _cases(torch, ms, eight, 77, 4, sizes=sizes)
        order = list(reversed(cases)) if how == 1 else cases
        if how == 2:
            for c in order:
                _step(ctx, ms, [c], 4)
        else:
            _step(ctx, ms, order, 4, table=how == 3)
        torch.cuda.synchronize()
        runs.append([x for c in cases for x in c.raw()])
    for other in runs[1:]:
        assert all(bool((x == y).all()) for x, y in zip(runs[0], other))


@pytest.mark.parametrize("eight", [False, True])
def test_special_values(ctx, torch, ms, eight):
    """Zeros, subnormals, values whose squares over- and underflow, infinities and NaN, each in a block of its own."""
    def change(p, g, m, v):
        k = g.size // 32
        for b in range(k):
            s = slice(32 * b, 32 * b + 32)
            if b == 0: g[s], m[s], v[s] = 0, 0, 0
            elif b == 1: g[s], m[s], v[s] = g[s] * 1e-22, m[s] * 1e-22, v[s] * 1e-40
            elif b == 2: g[s], m[s], v[s] = g[s] * 1e-30, 0, 0
            elif b == 3: g[32 * b + 5] = 1e25
            elif b == 4: g[32 * b + 6] = np.inf
            elif b == 5: g[32 * b + 7] = np.nan
            elif b == 6: g[32 * b + 8] = -np.inf
            elif b == 7: g[s], m[s], v[s] = g[s] * 1e12, m[s] * 1e12, v[s] * 1e24
            elif b == 8: g[s], m[s], v[s] = 0, m[s], v[s]
            elif b == 9: g[s], p[s] = -0.0, 0
            elif b == 10: m[32 * b + 3] = np.inf
            elif b == 11: v[32 * b + 3] = np.nan
            elif b == 12: g[s], m[s], v[s] = 3e-45, 0, 0
    for eps in (EPS, 0.0):
        cases = _cases(torch, ms, eight, 9, 3, sizes=(13 * 32 + 11,), change=change)
        _step(ctx, ms, cases, 3, eps=eps)
        torch.cuda.synchronize()
        for c in cases:
            c.check(3, eps=eps, what=f"eps {eps}")


def test_nan_blocks_stay_nan(ctx, torch, ms):
    """A gradient that is not finite makes its block's moment NaN; the other blocks go on."""
    rng = np.random.default_rng(3)
    c = Case(torch, ms, True, rng, 96, ("bf16", True, "f32"), 1)
    c.dg.t[40] = math.inf
    _step(ctx, ms, [c], 1)
    torch.cuda.synchronize()
    m, v = ms.adamw8_moments(tuple(d.t for d in c.ds))
    for x in (m, v):
        assert bool(x[32:64].isnan().all()) and bool(x[:32].isfinite().all()) and bool(x[64:].isfinite().all())
    c.dg.t[40] = 1.0
    _step(ctx, ms, [c], 2)
    torch.cuda.synchronize()
    w = to_np(c.dm.t)
    assert np.isnan(w[32:64]).all() and np.isfinite(np.delete(w, np.arange(32, 64))).all()


def test_foreign_state_bytes(ctx, torch, ms):
    """Every code and every exponent byte, as a state from elsewhere may hold them (e8m0 from 2^-127 on)."""
    n = 256 * 32
    rng = np.random.default_rng(12)
    c = Case(torch, ms, True, rng, n, ("f32", False, "f32"), 1)
    codes = rng.integers(0, 256, n).astype(np.uint8)
    c.state = (codes, np.arange(256, dtype=np.uint8), codes & 0x7F, np.arange(256, dtype=np.uint8)[::-1].copy())
    for d, x in zip(c.ds, c.state):
        d.t.copy_(torch.from_numpy(x))
    _step(ctx, ms, [c], 6)
    torch.cuda.synchronize()
    c.check(6, what="foreign state")


@pytest.mark.parametrize("eight", [False, True])
def test_offsets_past_32_bits(ctx, torch, ms, eight):
    """One tensor whose byte offsets pass 2^32 (and, with 8-bit moments, whose element numbers pass 2^34, where the
    random words take the number's upper half): windows at its start, at the borders and at its end."""
    n = (1 << 34) + 4101 if eight else (1 << 31) + 4101
    need = n * (8 if eight else 14)
    if torch.cuda.mem_get_info()[0] < 1.2 * need:
        pytest.skip("not enough device memory")
    windows = [0, (1 << 31) - 64, n - 4101 - 64] + ([(1 << 32) - 64, (1 << 33) - 64] if eight else [])
    size, step = 128, 2
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    if eight:
        state = ms.adamw8_state(p)
        desc = ms.adamw8_tensor(p, g, state)
    else:
        state = tuple(torch.zeros(n, device="cuda") for _ in range(2))
        desc = ms.adamw_mixed_tensor(p, g, *state)
    windows = sorted(set(windows)) + [n - 69]      # the last, partial block (of 5 elements) and the 64 before it
    rng = np.random.default_rng(2)
    host = []
    for at in windows:
        k = min(size, n - at)
        pw, gw = (_bf16((rng.standard_normal(k) * s).astype(np.float32)) for s in (0.02, 1.0))
        p[at:at + k] = torch.from_numpy(pw).bfloat16().cuda()
        g[at:at + k] = torch.from_numpy(gw).bfloat16().cuda()
        host.append((pw, gw))
    hp = ms.adamw_hparams(lr=LR, beta1=B1, beta2=B2, eps=EPS, weight_decay=WD, step=step)
    if eight:
        ctx.muon_adamw8_step([desc], hp, seed=SEED)
    else:
        ctx.muon_adamw_mixed_step([desc], hp)
    torch.cuda.synchronize()
    for at, (pw, gw) in zip(windows, host):
        k = len(pw)
        got = to_np(p[at:at + k])
        assert np.any(got != pw)
        if not eight:
            z = np.zeros(k, np.float32)
            ref = oracle.adamw_step_f32(pw, gw, z, z, LR, B1, B2, EPS, WD, step)
            assert_bitexact(got, _bf16(ref[0]), f"weights at {at}")
            assert_bitexact(to_np(state[0][at:at + k]), ref[1], f"exp_avg at {at}")
            assert_bitexact(to_np(state[1][at:at + k]), ref[2], f"exp_avg_sq at {at}")
            continue
        cut = at % 32           # a window may start inside a block
        m1 = (np.float32(1 - B1) * gw)
        v1 = (np.float32(1 - B2) * gw) * gw
        for x, floor, turn, (codes, scale) in ((m1, False, 0, state[:2]), (v1, True, 16, state[2:])):
            pad = np.concatenate([np.zeros(cut, np.float32), x])
            rc, re = oracle.quantise(pad, floor, np.arange(at - cut, at + k), SEED, step, turn)
            assert np.array_equal(codes[at:at + k].view(torch.uint8).cpu().numpy(), rc[cut:]), f"codes at {at}"
            b0 = (at - cut) // 32
            assert np.array_equal(scale[b0:b0 + len(re)].cpu().numpy(), re), f"scales at {at}"
    say(f"{n} elements: {len(windows)} windows")


def test_empty_calls(ctx, torch, ms):
    hp = ms.adamw_hparams()
    ctx.muon_adamw_mixed_step([], hp)
    ctx.muon_adamw8_step([], hp)
    e = torch.zeros(0, device="cuda")
    ctx.muon_adamw_mixed_step([ms.adamw_mixed_tensor(e, e, e, e)], hp)
    ctx.muon_adamw8_step([ms.adamw8_tensor(e, e, ms.adamw8_state(e))], hp)
    torch.cuda.synchronize()


@pytest.mark.parametrize("eight", [False, True])
def test_refused_call_writes_nothing(ctx, torch, ms, eight):
    cases = _cases(torch, ms, eight, 4, 2, sizes=(100,))
    before = [x for c in cases for x in c.raw()]
    for bad in ([cases[0], cases[1], cases[0]],):
        with pytest.raises(ms.MuonError) as err:
            _step(ctx, ms, bad, 2)
        assert err.value.status == ms.MUON_ERR_INVALID_ARGUMENT and "overlaps" in str(err.value)
    with pytest.raises(ms.MuonError):
        _step(ctx, ms, cases, 0)
    torch.cuda.synchronize()
    assert all(bool((x == y).all()) for x, y in zip(before, [x for c in cases for x in c.raw()]))


# ----------------------------------------------------------------------------------------------- gradient norm

def _norm(torch, ctx, ms, grads, max_norm=1.0, stream=None):
    norm = torch.full((3,), -1.0, dtype=torch.float64, device="cuda")
    factor = torch.full((3,), -1.0, device="cuda")
    ctx.muon_grad_norm(grads, max_norm, norm[1:2], factor[1:2], stream)
    torch.cuda.synchronize()
    n, f = norm.cpu().numpy(), factor.cpu().numpy()
    assert n[0] == n[2] == -1 and f[0] == f[2] == -1
    return n[1], f[1]


# fp64 sums: no value passes through more than a few thousand additions, 2^-53 each, before the square root
NORM_TOL = 1e-12


def _check_norm(got, host, max_norm, what):
    n, f = oracle.grad_norm(host, max_norm)
    if not math.isfinite(n):
        assert (math.isnan(got[0]) and math.isnan(n)) or got[0] == n, what
        assert math.isnan(got[1]), what
        return
    assert abs(got[0] - n) <= NORM_TOL * n, what
    assert abs(float(got[1]) - float(f)) <= 2.0 ** -23 * float(f), what   # one fp32 rounding of a quotient each


@pytest.mark.parametrize("shift", [0, 1, 2, 4])
@pytest.mark.parametrize("gd", ["f32", "bf16"])
def test_grad_norm_sizes(ctx, torch, ms, gd, shift):
    """Each size alone, all of them together, and 300 tensors in one call (more than one launch takes)."""
    rng = np.random.default_rng(31)
    every = []
    for n in SIZES + (8191, 8192, 8193, 300001):
        x = (rng.standard_normal(n) * np.exp(3 * rng.standard_normal(n))).astype(np.float32)
        x = _bf16(x) if gd == "bf16" else x
        d = Guarded(torch, x, _dtype(torch, gd), shift)
        every.append((x, d))
        _check_norm(_norm(torch, ctx, ms, [ms.grad(d.t)]), [x], 1.0, f"n={n}")
    for max_norm in (1e-3, 1.0, 1e6, math.inf):
        _check_norm(_norm(torch, ctx, ms, [ms.grad(d.t) for _, d in every], max_norm), [x for x, _ in every], max_norm,
                    f"all, max_norm {max_norm}")
    many = (every * 13)[:300]
    _check_norm(_norm(torch, ctx, ms, ms.table(ms.grad(d.t) for _, d in many)), [x for x, _ in many], 1.0, "300")
    for x, d in every:
        d.check("gradient")
        assert_bitexact(d.np(), x, "a gradient is only read")


def test_grad_norm_mixed_types_and_extremes(ctx, torch, ms):
    rng = np.random.default_rng(32)
    a = rng.standard_normal(5000).astype(np.float32)
    b = _bf16(rng.standard_normal(3001).astype(np.float32))
    ta, tb = torch.from_numpy(a).cuda(), torch.from_numpy(b).bfloat16().cuda()
    _check_norm(_norm(torch, ctx, ms, [ms.grad(ta), ms.grad(tb)]), [a, b], 1.0, "mixed types")
    for s in (1e30, 1e-30, 1e-42):       # squares far outside fp32
        x = (a * np.float32(s)).astype(np.float32)
        _check_norm(_norm(torch, ctx, ms, [ms.grad(torch.from_numpy(x).cuda())]), [x], 1.0, f"scale {s}")
    assert _norm(torch, ctx, ms, []) == (0.0, 1.0)
    assert _norm(torch, ctx, ms, [ms.grad(torch.zeros(0, device="cuda"))]) == (0.0, 1.0)
    assert _norm(torch, ctx, ms, [ms.grad(torch.zeros(100, device="cuda"))]) == (0.0, 1.0)
    one = torch.ones(1, device="cuda")
    assert _norm(torch, ctx, ms, [ms.grad(one)]) == (1.0, 1.0)          # not above max_norm
    assert _norm(torch, ctx, ms, [ms.grad(one), ms.grad(one), ms.grad(one), ms.grad(one)]) == (2.0, 0.5)
    for bad in (math.inf, -math.inf, math.nan):
        x = a.copy()
        x[4321] = bad
        _check_norm(_norm(torch, ctx, ms, [ms.grad(tb), ms.grad(torch.from_numpy(x).cuda())]), [b, x], 1.0, str(bad))
    again = [_norm(torch, ctx, ms, [ms.grad(ta), ms.grad(tb)]) for _ in range(5)]
    assert len(set(again)) == 1, "the same bits every time"


def test_grad_norm_large(ctx, torch, ms):
    """Past 2^32 bytes and past the workgroups of one launch; each window counts once."""
    n = (1 << 31) + 12345
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    total = 0.0
    for at in (0, 12345678, (1 << 31) - 1, n - 1):
        g[at] = 3.0
        total += 9.0
    assert _norm(torch, ctx, ms, [ms.grad(g)], 100.0) == (math.sqrt(total), 1.0)
    g.fill_(0.5)
    norm, _ = _norm(torch, ctx, ms, [ms.grad(g)])
    assert norm == math.sqrt(n * 0.25)   # every partial sum is exact


def test_grad_norm_many_tables(torch, ms):
    """More tensors than the sums' memory holds tables of, eager and captured: the sums are joined on the way, and the
    last, small table joins what is left.  Multiples of 1/8 below 2^7, so every partial sum is exact."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(33)
    x = torch.randint(-500, 501, (32768,), generator=gen, device="cuda") / 8.0      # four chunks
    last = torch.full((3,), 2.0, device="cuda")
    count = 17 * 256 + 2
    ctxs = ms.Context(0), ms.Context(0)
    try:
        grads = ms.table([ms.grad(x)] * count + [ms.grad(last)])

        def expected():
            return math.sqrt(count * float((x.double() ** 2).sum()) + float((last.double() ** 2).sum()))

        assert _norm(torch, ctxs[0], ms, grads)[0] == expected()
        norm, factor = torch.zeros(1, dtype=torch.float64, device="cuda"), torch.zeros(1, device="cuda")
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            ctxs[1].muon_grad_norm(grads, 1.0, norm, factor, torch.cuda.current_stream())
        for k in range(3):
            x.mul_(0.5)
            graph.replay()
            eager = _norm(torch, ctxs[0], ms, grads)
            assert (float(norm), np.float32(float(factor))) == eager and eager[0] == expected(), f"replay {k}"
    finally:
        torch.cuda.synchronize()
        for c in ctxs:
            c.close()


# -------------------------------------------------------------------------------- muon_step with the clip factor

@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("gd", ["f32", "bf16"])
def test_muon_step_with_factor(ctx, torch, ms, gd, shift):
    """The momentum is that of gradients multiplied beforehand, bit for bit, in both orientations, vector widths and
    entry points; a factor of 1 and no factor give the same bits."""
    rng = np.random.default_rng(41)
    f = np.float32(0.37)
    tf = torch.tensor([float(f)], device="cuda")
    shapes = [(64, 128), (128, 64), (33, 65), (65, 33), (200, 300)]
    for entry in ("muon_step", "muon_step_noalloc"):
        dev, host = [], []
        for rows, cols in shapes:
            g = rng.standard_normal((rows, cols)).astype(np.float32)
            g = _bf16(g) if gd == "bf16" else g
            m = rng.standard_normal((rows, cols)).astype(np.float32)
            w = _bf16((rng.standard_normal((rows, cols)) * 0.02).astype(np.float32))
            host.append((w, g, m))
            runs = []
            for _ in range(3):
                t = [Guarded(torch, x.ravel(), d, shift).t.view(rows, cols)
                     for x, d in ((w, torch.bfloat16), (g, _dtype(torch, gd)), (m, torch.float32))]
                runs.append(t + [torch.empty(rows, cols, device="cuda")])
            dev.append(runs)
        for k, factor in enumerate((tf, None, torch.ones(1, device="cuda"))):
            getattr(ctx, entry)([ms.matrix(*d[k]) for d in dev], ms.make_hparams(grad_factor=factor))
        torch.cuda.synchronize()
        for (w, g, m), runs in zip(host, dev):
            m_ref, n_ref = oracle.nesterov_momentum_f32(m, f * g, 0.95)
            assert_bitexact(to_np(runs[0][2]), m_ref, f"{entry} momentum {w.shape}")
            ref = oracle.muon_step(w, f * g, m, param_bf16=True)
            x = to_np(runs[0][3])
            assert rel_fro(x * math.sqrt(max(w.shape)) * 0.2, ref["o"]) <= BF16_TOL
            for x, y in zip(runs[1], runs[2]):
                assert_bitexact(to_np(x), to_np(y), f"{entry}: factor 1 and none")


def _sequence(torch, ms, ctx, t, step, stream=None):
    """Clip, Muon and both AdamW steps, as a training step has them."""
    ctx.muon_grad_norm(t["grads"], 1.0, t["norm"], t["factor"], stream)
    ctx.muon_step(t["mats"], t["hp"], stream)
    hp = ms.adamw_hparams(lr=LR, beta1=B1, beta2=B2, eps=EPS, weight_decay=WD, step=step)
    ctx.muon_adamw_mixed_step(t["mixed"], hp, grad_factor=t["factor"], stream=stream)
    ctx.muon_adamw8_step(t["eight"], hp, seed=SEED, grad_factor=t["factor"], stream=stream)


def _model(torch, ms, seed):
    """A small model's tensors: two matrices for Muon, a head with a master copy, an embedding with 8-bit moments and
    a few norm weights."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    bf = torch.bfloat16
    t = {"keep": [], "state": []}

    def new(*shape, scale=1.0, dtype=bf):
        x = (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)
        t["keep"].append(x)
        return x

    t["norm"] = torch.zeros(1, dtype=torch.float64, device="cuda")
    t["factor"] = torch.zeros(1, device="cuda")
    t["g"], mats, mixed, eight = [], [], [], []
    for rows, cols in ((128, 256), (256, 128)):
        p, g, m = new(rows, cols, scale=0.02), new(rows, cols), new(rows, cols, scale=0, dtype=torch.float32)
        mats.append(ms.matrix(p, g, m))
        t["g"].append(g)
        t["state"] += [p, m]
    for n in (500 * 64, 64, 64, 65):
        p, g, m, v = new(n, scale=0.02), new(n), new(n, scale=0, dtype=torch.float32), new(n, scale=0, dtype=torch.float32)
        w = p.float()
        t["keep"].append(w)
        mixed.append(ms.adamw_mixed_tensor(p, g, m, v, master=w))
        t["g"].append(g)
        t["state"] += [p, m, v, w]
    p, g = new(501, 64, scale=0.02), new(501, 64)
    s = ms.adamw8_state(p)
    eight.append(ms.adamw8_tensor(p, g, s))
    t["g"].append(g)
    t["state"] += [p] + [x.view(torch.uint8) for x in s]
    t["grads"] = ms.table(ms.grad(x) for x in t["g"])
    t["mats"], t["mixed"], t["eight"] = mats, ms.table(mixed), ms.table(eight)
    t["hp"] = ms.make_hparams(grad_factor=t["factor"])
    return t


def test_run_together_against_oracle(ctx, torch, ms):
    """Clip, Muon, AdamW with 32-bit and with 8-bit moments, two steps, each against the oracle from the clipped
    gradients."""
    t = _model(torch, ms, 5)
    host = [to_np(x) if x.dtype != torch.uint8 else x.cpu().numpy() for x in t["state"]]
    for step in (1, 2):
        _sequence(torch, ms, ctx, t, step)
        torch.cuda.synchronize()
        grads = [to_np(g).reshape(-1) for g in t["g"]]
        norm, f = oracle.grad_norm(grads, 1.0)
        assert abs(float(t["norm"]) - norm) <= NORM_TOL * norm
        f_gpu = np.float32(float(t["factor"]))
        assert abs(float(f_gpu) - float(f)) <= 2.0 ** -23 * float(f)
        now = [to_np(x) if x.dtype != torch.uint8 else x.cpu().numpy() for x in t["state"]]
        for i in range(2):
            g = f_gpu * to_np(t["g"][i])
            m_ref, _ = oracle.nesterov_momentum_f32(host[2 * i + 1], g, 0.95)
            assert_bitexact(now[2 * i + 1], m_ref, f"step {step} momentum {i}")
        for i in range(4):
            p, m, v, w = host[4 + 4 * i:8 + 4 * i]
            rp, rm, rv = oracle.adamw_step_f32(w, f_gpu * grads[2 + i], m, v, LR, B1, B2, EPS, WD, step)
            got = now[4 + 4 * i:8 + 4 * i]
            for x, ref, what in zip(got, (_bf16(rp), rm, rv, rp), ("param", "exp_avg", "exp_avg_sq", "master")):
                assert_bitexact(x, ref, f"step {step} tensor {i} {what}")
        p, *s = host[20:]
        s = [x.reshape(-1) for x in s]
        ref, update, rs = oracle.adamw8_step(p.reshape(-1), grads[6], s, LR, B1, B2, EPS, WD, step, SEED, f_gpu)
        for x, y in zip(now[21:], rs):
            assert np.array_equal(x.reshape(-1), y)
        err = np.abs(now[20].reshape(-1) - ref)
        assert np.all(err <= 2.0 ** -20 * np.abs(update) + (2.0 ** -22 + 2.0 ** -8) * np.maximum(np.abs(ref), np.abs(p.reshape(-1))))
        host = now
        for g in t["g"]:
            g.mul_(1.5)


def test_run_together_captured(torch, ms):
    """The same run captured into a graph on the context's first calls of these entry points, replayed with other
    gradients each time and eager work of another context between, against eager runs."""
    graph_ctx, eager_ctx, between_ctx = ms.Context(0), ms.Context(0), ms.Context(0)
    try:
        a, b, other = _model(torch, ms, 6), _model(torch, ms, 6), _model(torch, ms, 7)
        side = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()

        def run(c, t, step):
            ctx_stream = torch.cuda.current_stream()
            c.muon_grad_norm(t["grads"], 1.0, t["norm"], t["factor"], ctx_stream)
            hp = ms.adamw_hparams(lr=LR, beta1=B1, beta2=B2, eps=EPS, weight_decay=WD, step=step)
            c.muon_adamw_mixed_step(t["mixed"], hp, grad_factor=t["factor"])
            c.muon_adamw8_step(t["eight"], hp, seed=SEED, grad_factor=t["factor"])

        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            run(graph_ctx, a, 3)
        start = [x.clone() for x in a["state"]]
        for x, y in zip(start, b["state"]):
            assert bool((x.view(torch.uint8) == y.view(torch.uint8)).all()), "a capture runs nothing"
        for k in range(4):
            for x, y in zip(a["g"], b["g"]):
                x.mul_(0.9 + 0.1 * k)
                y.copy_(x)
            graph.replay()
            run(between_ctx, other, 1 + k)
            run(eager_ctx, b, 3)
            torch.cuda.synchronize()
            assert float(a["norm"]) == float(b["norm"]) and float(a["factor"]) == float(b["factor"])
            for x, y in zip(a["state"], b["state"]):
                assert bool((x.view(torch.uint8) == y.view(torch.uint8)).all()), f"replay {k}"
    finally:
        torch.cuda.synchronize()
        for c in (graph_ctx, eager_ctx, between_ctx):
            c.close()


def test_other_stream(ctx, torch, ms):
    """Two streams, each with tensors and a context of its own, at the same time; the results are those of the
    current stream."""
    runs = []
    ctxs = [ms.Context(0), ms.Context(0)]
    try:
        ts = [_model(torch, ms, 8) for _ in range(3)]
        _sequence(torch, ms, ctx, ts[2], 1)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for c, t, s in zip(ctxs, ts, streams):
            _sequence(torch, ms, c, t, 1, s)
        torch.cuda.synchronize()
        for t in ts[:2]:
            for x, y in zip(t["state"], ts[2]["state"]):
                runs.append(bool((x.contiguous().view(torch.uint8) == y.contiguous().view(torch.uint8)).all()))
        assert all(runs)
    finally:
        torch.cuda.synchronize()
        for c in ctxs:
            c.close()


def test_profile_stages(ctx, torch, ms):
    t = _model(torch, ms, 9)
    ctx.muon_profile_enable(True)
    try:
        _sequence(torch, ms, ctx, t, 1)
        torch.cuda.synchronize()
        st = ctx.muon_profile_read()
    finally:
        ctx.muon_profile_enable(False)
    n = sum(x.numel() for x in t["g"])
    assert st["grad_norm"]["bytes"] == 2 * n
    assert st["adamw_mixed"]["bytes"] == (500 * 64 + 64 + 64 + 65) * (16 + 2 + 8 + 2)
    assert st["adamw8"]["bytes"] == 501 * 64 * (4 + 4 / 32 + 2 + 4)
