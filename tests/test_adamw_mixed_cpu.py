"""What the mixed-type AdamW steps and the gradient norm refuse, their structures' layout, and the pins of the 8-bit
oracle; needs no GPU."""

import ctypes
import math
import os
import subprocess

import numpy as np
import pytest

import muon_step_amd as ms
import oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 1 << 40   # fake device addresses: validation never dereferences them
F32, BF16 = ms.MUON_F32, ms.MUON_BF16


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ms.LIB_PATH):
        pytest.fail("libmuon_step.so is not built (run __graft_entry__.build())")
    return ms.load()


def test_struct_layouts_match_header(tmp_path):
    kinds = (ms.muon_adamw_mixed_tensor, ms.muon_adamw8_tensor, ms.muon_grad, ms.muon_hparams)
    body = "".join(f'printf("{k.__name__} %zu\\n", sizeof({k.__name__}));' +
                   "".join(f'printf("{k.__name__}.{f[0]} %zu\\n", offsetof({k.__name__}, {f[0]}));' for f in k._fields_)
                   for k in kinds)
    src = tmp_path / "layout.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"muon_step.h\"\nint main(void) {" + body +
                   f'printf("block %d\\n", MUON_ADAMW8_BLOCK); return 0; }}')
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe],
                   check=True)
    got = dict(line.rsplit(" ", 1) for line in
               subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines())
    for k in kinds:
        assert int(got[k.__name__]) == ctypes.sizeof(k)
        for f in k._fields_:
            assert int(got[f"{k.__name__}.{f[0]}"]) == getattr(k, f[0]).offset, f
    assert int(got["block"]) == ms.MUON_ADAMW8_BLOCK == oracle.adamw8.BLOCK


# ------------------------------------------------------------------------------------------------ refusals

def _mixed(i=0, n=1000, pd=BF16, gd=BF16, master=False):
    o = BASE + i * (1 << 40)
    return ms.muon_adamw_mixed_tensor(o, o + (1 << 32) if master else None, o + (2 << 32), o + (3 << 32),
                                      o + (4 << 32), n, pd, gd)


def _eight(i=0, n=1000, pd=BF16, gd=BF16, master=False):
    o = BASE + i * (1 << 40)
    return ms.muon_adamw8_tensor(o, o + (1 << 32) if master else None, o + (2 << 32), o + (3 << 32), o + (4 << 32),
                                 o + (5 << 32), o + (6 << 32), n, pd, gd)


def _check(lib, ts, hp=None, factor=None, count=None, hp_null=False):
    kind = type(ts[0])
    arr = (kind * len(ts))(*ts)
    fn = lib.muon_check_adamw_mixed_args if kind is ms.muon_adamw_mixed_tensor else lib.muon_check_adamw8_args
    buf = ctypes.create_string_buffer(512)
    hp = hp or ms.adamw_hparams()
    st = fn(arr, len(ts) if count is None else count, None if hp_null else ctypes.byref(hp), factor, buf, 512)
    return st, buf.value.decode()


@pytest.mark.parametrize("make", [_mixed, _eight])
def test_adamw_accepts(lib, make):
    ok = (ms.MUON_OK, "")
    for pd, gd, master in ((F32, F32, False), (F32, BF16, False), (BF16, F32, True), (BF16, BF16, True),
                           (BF16, F32, False), (BF16, BF16, False)):
        assert _check(lib, [make(0, 1000, pd, gd, master), make(1, 1, pd, gd, master)], factor=BASE - 4) == ok
    assert _check(lib, [make(), make(1)], count=0) == ok
    empty = type(make())(numel=0)   # the pointers of an empty tensor are not looked at
    assert _check(lib, [empty, make()]) == ok
    a, b = make(0), make(1)
    b.grad = a.grad                 # gradients may share memory
    assert _check(lib, [a, b]) == ok
    a = make(0)
    a.grad = a.param + 2000         # starts where param ends
    assert _check(lib, [a]) == ok
    assert _check(lib, [make()], hp=ms.adamw_hparams(beta1=0.0, beta2=0.0, eps=0.0)) == ok


@pytest.mark.parametrize("make", [_mixed, _eight])
@pytest.mark.parametrize("case", ["param", "grad", "exp_avg", "exp_avg_sq", "numel_neg", "numel_big", "param_dtype",
                                  "grad_dtype", "master_f32", "odd_param", "odd_grad", "odd_master", "same_twice",
                                  "grad_in_param", "grad_in_master", "moments_share", "factor_odd", "factor_in_param",
                                  "lr", "wd", "eps_neg", "eps_nan", "beta1_one", "beta1_neg", "beta2_one", "beta2_nan",
                                  "step0", "hp_null", "count_neg", "count_big"])
def test_adamw_refuses(lib, make, case):
    a, b = make(0, master=True), make(1)
    hp, kw = ms.adamw_hparams(), {}
    if case in ("param", "grad", "exp_avg", "exp_avg_sq"): setattr(a, case, None)
    elif case == "numel_neg": a.numel = -1
    elif case == "numel_big": a.numel = (1 << 38) + 1
    elif case == "param_dtype": a.param_dtype = 7
    elif case == "grad_dtype": a.grad_dtype = -1
    elif case == "master_f32": a.param_dtype = F32
    elif case == "odd_param": a.param += 1
    elif case == "odd_grad": a.grad += 1
    elif case == "odd_master": a.master += 2
    elif case == "same_twice": b = a
    elif case == "grad_in_param": b.grad = a.param + 8
    elif case == "grad_in_master": b.grad = a.master + 3998
    elif case == "moments_share": a.exp_avg_sq = a.exp_avg
    elif case == "factor_odd": kw["factor"] = BASE - 6
    elif case == "factor_in_param": kw["factor"] = a.param + 1996
    elif case == "lr": hp.lr = math.inf
    elif case == "wd": hp.weight_decay = math.nan
    elif case == "eps_neg": hp.eps = -1e-8
    elif case == "eps_nan": hp.eps = math.nan
    elif case == "beta1_one": hp.beta1 = 1.0
    elif case == "beta1_neg": hp.beta1 = -0.1
    elif case == "beta2_one": hp.beta2 = 1.0
    elif case == "beta2_nan": hp.beta2 = math.nan
    elif case == "step0": hp.step = 0
    elif case == "hp_null": kw["hp_null"] = True
    elif case == "count_neg": kw["count"] = -1
    elif case == "count_big": kw["count"] = 1 << 31
    st, msg = _check(lib, [a, b], hp=hp, **kw)
    assert st == ms.MUON_ERR_INVALID_ARGUMENT and msg


def test_adamw8_refuses_more(lib):
    for field in ("exp_avg_scale", "exp_avg_sq_scale"):
        a = _eight()
        setattr(a, field, None)
        assert _check(lib, [a])[0] == ms.MUON_ERR_INVALID_ARGUMENT
    a = _eight(n=1000)                       # 32 scale bytes
    a.exp_avg_sq_scale = a.exp_avg_scale + 31
    st, msg = _check(lib, [a])
    assert st == ms.MUON_ERR_INVALID_ARGUMENT and "scale" in msg
    a.exp_avg_sq_scale = a.exp_avg_scale + 32
    assert _check(lib, [a]) == (ms.MUON_OK, "")
    assert _check(lib, [_eight()], hp=ms.adamw_hparams(eps=1e-39))[0] == ms.MUON_ERR_INVALID_ARGUMENT
    assert _check(lib, [_mixed()], hp=ms.adamw_hparams(eps=1e-39))[0] == ms.MUON_OK


@pytest.mark.parametrize("eight", [False, True])
def test_overlap_check_against_brute_force(lib, eight):
    """Random layouts of a few dozen tensors, in and out of address order, some with one range moved onto another's
    last or first byte: refused exactly where two ranges share a byte and one of them is written."""
    rng = np.random.default_rng(4)
    fields = (["param", "master", "grad", "exp_avg", "exp_avg_sq"] +
              (["exp_avg_scale", "exp_avg_sq_scale"] if eight else []))
    refused = 0
    for trial in range(300):
        count = int(rng.integers(1, 30))
        ts = []
        for _ in range(count):
            t = (ms.muon_adamw8_tensor if eight else ms.muon_adamw_mixed_tensor)()
            t.numel = int(rng.choice([0, 1, 31, 32, 33, 1000]))
            t.param_dtype, t.grad_dtype = BF16, int(rng.integers(0, 2))
            ts.append(t)
        has_master = rng.random(count) < 0.5

        def size(t, f):
            if f == "param": return 2 * t.numel
            if f == "grad": return (2 if t.grad_dtype == BF16 else 4) * t.numel
            if f.endswith("scale"): return -(-t.numel // 32)
            return t.numel if eight and f != "master" else 4 * t.numel

        slots = [(i, f) for i in range(count) for f in fields if f != "master" or has_master[i]]
        if trial % 2: rng.shuffle(slots)
        at = BASE
        for i, f in slots:
            setattr(ts[int(i)], str(f), at)
            at += -(-size(ts[int(i)], str(f)) // 4) * 4 + int(rng.choice([0, 0, 4, 64]))
        if trial % 3 == 0:                       # move one range to another's end or start
            (i, f), (j, h) = (slots[k] for k in rng.integers(0, len(slots), 2))
            i, f, j, h = int(i), str(f), int(j), str(h)
            addr = getattr(ts[j], h) + int(rng.choice([0, max(0, size(ts[j], h) - 4), size(ts[j], h)]))
            setattr(ts[i], f, -(-addr // 4) * 4)
        spans = [(getattr(ts[int(i)], str(f)), size(ts[int(i)], str(f)), f != "grad") for i, f in slots]
        spans = [s for s in spans if s[1] > 0]
        hit = any(a[0] < b[0] + b[1] and b[0] < a[0] + a[1] and (a[2] or b[2])
                  for k, a in enumerate(spans) for b in spans[:k])
        st, msg = _check(lib, ts)
        assert st == (ms.MUON_ERR_INVALID_ARGUMENT if hit else ms.MUON_OK), (trial, msg)
        assert ("overlaps" in msg) == hit
        refused += hit
    assert 20 < refused < 200


def test_grad_norm_refuses(lib):
    g = ms.muon_grad(BASE, 1000, BF16, 0)
    norm, factor = BASE - 16, BASE - 8

    def check(gs, max_norm=1.0, norm=norm, factor=factor, count=None):
        arr = (ms.muon_grad * max(1, len(gs)))(*gs)
        buf = ctypes.create_string_buffer(512)
        st = lib.muon_check_grad_norm_args(arr, len(gs) if count is None else count, max_norm, norm, factor, buf, 512)
        assert (st == ms.MUON_OK) == (buf.value == b"")
        return st

    bad = ms.MUON_ERR_INVALID_ARGUMENT
    assert check([g]) == ms.MUON_OK
    assert check([g, g]) == ms.MUON_OK       # the same gradient twice counts twice
    assert check([]) == ms.MUON_OK
    assert check([ms.muon_grad(None, 0, F32, 0)]) == ms.MUON_OK
    assert check([g], max_norm=math.inf) == ms.MUON_OK
    for m in (0.0, -1.0, math.nan):
        assert check([g], max_norm=m) == bad
    assert check([g], norm=None) == bad
    assert check([g], factor=None) == bad
    assert check([g], norm=norm + 4) == bad
    assert check([g], factor=factor + 2) == bad
    assert check([g], factor=norm + 4) == bad             # overlaps norm
    assert check([g], norm=BASE + 992) == bad             # inside the gradient
    assert check([g], factor=BASE + 1996) == bad
    assert check([g], factor=BASE + 2000) == ms.MUON_OK   # behind it
    assert check([ms.muon_grad(BASE, -1, F32, 0)]) == bad
    assert check([ms.muon_grad(BASE, (1 << 40) + 1, F32, 0)]) == bad
    assert check([ms.muon_grad(BASE, 8, 3, 0)]) == bad
    assert check([ms.muon_grad(BASE + 2, 8, F32, 0)]) == bad
    assert check([ms.muon_grad(None, 8, F32, 0)]) == bad
    assert check([g], count=-1) == bad


def test_step_refuses_factor(lib):
    hp = ms.make_hparams()
    m = ms.muon_matrix(BASE, BASE + (1 << 30), BASE + (2 << 30), None, 64, 128, BF16, BF16)
    arr = (ms.muon_matrix * 1)(m)

    def check():
        return lib.muon_check_step_args(arr, 1, ctypes.byref(hp), None, 0)

    assert check() == ms.MUON_OK
    hp.grad_factor = BASE - 4
    assert check() == ms.MUON_OK
    hp.grad_factor = BASE - 2
    assert check() == ms.MUON_ERR_INVALID_ARGUMENT
    hp.grad_factor = BASE + (2 << 30) + 16   # in the momentum, which the step writes
    assert check() == ms.MUON_ERR_INVALID_ARGUMENT
    hp.grad_factor = BASE + (1 << 30)        # in the gradient, which it only reads
    assert check() == ms.MUON_OK


def test_null_context(lib):
    a = ms.MUON_ERR_INVALID_ARGUMENT
    assert lib.muon_adamw_mixed_step(None, None, 0, None, None, None) == a
    assert lib.muon_adamw8_step(None, None, 0, None, 0, None, None) == a
    assert lib.muon_grad_norm(None, None, 0, 1.0, None, None, None) == a


def test_binding_refuses_before_any_launch():
    import torch
    f, b = torch.zeros(64), torch.zeros(64, dtype=torch.bfloat16)
    state = ms.adamw8_state(b)
    assert [t.dtype for t in state] == [torch.float8_e4m3fn, torch.uint8] * 2
    assert [t.numel() for t in state] == [64, 2, 64, 2]
    with pytest.raises(TypeError, match="bfloat16 param"):
        ms.adamw_mixed_tensor(f, f, f, f, master=f)
    with pytest.raises(TypeError, match="master must be float32"):
        ms.adamw_mixed_tensor(b, b, f, f, master=b)
    with pytest.raises(TypeError, match="exp_avg must be float32"):
        ms.adamw_mixed_tensor(b, b, b, f)
    with pytest.raises(TypeError, match="unsupported dtype"):
        ms.adamw_mixed_tensor(b.half(), b, f, f)
    with pytest.raises(ValueError, match="grad must be contiguous"):
        ms.adamw_mixed_tensor(b, torch.zeros(128, dtype=torch.bfloat16)[::2], f, f)
    with pytest.raises(ValueError, match="exp_avg_sq must be contiguous"):
        ms.adamw_mixed_tensor(b, b, f, torch.zeros(63))
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        ms.adamw_mixed_tensor(b, b, f, f)
    with pytest.raises(ValueError, match="exp_avg_scale must be contiguous, with 2"):
        ms.adamw8_tensor(b, b, (state[0], torch.zeros(3, dtype=torch.uint8), state[2], state[3]))
    with pytest.raises(TypeError, match="exp_avg_sq must be one of"):
        ms.adamw8_tensor(b, b, (state[0], state[1], f, state[3]))
    with pytest.raises(ValueError, match="state must hold"):
        ms.adamw8_tensor(b, b, state[:3])
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        ms.adamw8_tensor(b, b, state)
    with pytest.raises(ValueError, match="contiguous"):
        ms.grad(torch.zeros(4, 4).t())
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        ms.grad(f)
    with pytest.raises(TypeError, match="one float32 element"):
        ms.make_hparams(grad_factor=torch.zeros(2))
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        ms.make_hparams(grad_factor=torch.zeros(1))
    ctx = ms.Context.__new__(ms.Context)   # no device context: the checks come first
    ctx.lib, ctx.device, ctx.handle = ms.load(), 0, None
    hp = ms.adamw_hparams()
    with pytest.raises(TypeError, match="expected a muon_adamw8_tensor"):
        ctx.muon_adamw8_step([_mixed()], hp)
    with pytest.raises(TypeError, match="expected a table of muon_grad"):
        ctx._check_tensors = lambda named: None
        ctx.muon_grad_norm(ms.table([_eight()]), 1.0, torch.zeros(1, dtype=torch.float64), torch.zeros(1))
    del ctx._check_tensors
    with pytest.raises(ValueError, match="seed"):
        ctx.muon_adamw8_step([_eight()], hp, seed=-1)
    with pytest.raises(TypeError, match="norm must be one float64"):
        ctx.muon_grad_norm([], 1.0, torch.zeros(1), torch.zeros(1))
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        ctx.muon_grad_norm([], 1.0, torch.zeros(1, dtype=torch.float64), torch.zeros(1))
    t = _mixed()
    t._device = 3
    with pytest.raises(ValueError, match="cuda:3"):
        ctx.muon_adamw_mixed_step([t], hp)
    with pytest.raises(ValueError, match="cuda:3"):
        ctx.muon_adamw_mixed_step(ms.table([t]), hp)
    u = _mixed(1)
    u._device = 0
    with pytest.raises(ValueError, match="several GPUs"):
        ms.table([t, u])


# ------------------------------------------------------------------------------------------------ oracle pins

def test_oracle_code_values_match_torch():
    import torch
    ours = oracle.e4m3_values()
    theirs = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ours, theirs, equal_nan=True)
    e = torch.arange(256, dtype=torch.uint8)
    scales = e.view(torch.float8_e8m0fnu).double().numpy()
    got = oracle.moment_values(np.full(256 * 32, 0x38, np.uint8), e.numpy())[::32]   # 0x38 is 1
    assert np.array_equal(got, scales, equal_nan=True)


def test_oracle_adamw8_weights_match_torch_adamw():
    """From moments that 8 bits hold exactly, one step in float64 against torch's AdamW."""
    import torch
    r = np.random.default_rng(3)
    n = 256
    state = (r.integers(0, 127, n).astype(np.uint8), np.full(8, 118, np.uint8),
             r.integers(1, 127, n).astype(np.uint8), np.full(8, 112, np.uint8))
    p, g = r.standard_normal(n).astype(np.float32), r.standard_normal(n).astype(np.float32)
    got, _, _ = oracle.adamw8_step(p, g, state, 0.02, 0.9, 0.95, 1e-8, 0.1, 5)
    t = torch.tensor(p, dtype=torch.float64, requires_grad=True)
    opt = torch.optim.AdamW([t], lr=0.02, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    opt.state[t] = {"step": torch.tensor(4.0), "exp_avg": torch.tensor(oracle.moment_values(state[0], state[1])),
                    "exp_avg_sq": torch.tensor(oracle.moment_values(state[2], state[3]))}
    t.grad = torch.tensor(g, dtype=torch.float64)
    opt.step()
    # the moments' three fp32 roundings: at most 3 x 2^-24 of the sums' absolute terms
    assert np.allclose(got, t.detach().numpy(), rtol=0, atol=1e-6)


def test_oracle_exponents():
    """The block exponent is the smallest that brings the largest magnitude to 448 or less."""
    for a in (448.0, 448.0001, 447.9, 1.0, 0.875, 0.8751, 3e-20, 3.4e38, 2.0 ** -126, 1e-45, 0.0):
        x = np.zeros(32, np.float32)
        x[7] = a
        e = int(oracle.quantise(x, False, np.arange(32), 0, 1, 0)[1][0])
        y = math.ldexp(float(x[7]), 127 - e)
        assert y <= 448
        assert e == 17 or 2 * y > 448
    codes, e = oracle.quantise(np.array([1.0, np.inf, 0.0], np.float32), False, np.arange(3), 0, 1, 0)
    assert e[0] == 255 and np.all(codes == 0x7F)
    assert np.isnan(oracle.moment_values(codes, e)).all()


@pytest.mark.parametrize("floor", [False, True])
def test_oracle_rounding_is_unbiased(floor):
    """Of 4096 equal values, 16 steps each, the share that is rounded up is the value's place between the two codes.
    The elements of a group of four share a word: at least 16384 independent draws, whose mean has a standard
    deviation of at most 0.5 / 128; the bound is five of them."""
    n = 4096
    for place, low in ((0.25, 0.5), (0.9, 0.5), (0.03, 3 * 2.0 ** -9), (0.5, 2.0 ** -6)):
        x = np.full(n, 448.0, np.float32)
        gap = 0.0625 if low == 0.5 else 2.0 ** -9
        x[np.arange(n) % 32 != 0] = low + place * gap
        up = []
        for step in range(1, 17):
            codes, e = oracle.quantise(x, floor, np.arange(n), 77, step, 16 if floor else 0)
            assert np.all(e == 127)
            v = oracle.moment_values(codes, e)[np.arange(n) % 32 != 0]
            assert set(np.unique(v)) <= {low, low + gap}
            up.append(np.mean(v > low))
        assert abs(np.mean(up) - place) <= 5 * 0.5 / 128


def test_oracle_floor():
    """A second moment is never rounded to zero beside one above zero; alone it stays zero."""
    x = np.zeros(64, np.float32)
    x[:3] = [1.0, 1e-12, 0.0]
    codes, e = oracle.quantise(x, True, np.arange(64), 0, 1, 16)
    assert np.all(codes[:32] >= 1) and np.all(codes[32:] == 0)
    v = oracle.moment_values(codes, e)
    assert v[1] == v[2] == 2.0 ** (int(e[0]) - 127 - 9)


def test_oracle_dither_spreads():
    u = oracle.dither(np.arange(1 << 16), 5, 9, 0)
    w = oracle.dither(np.arange(1 << 16), 5, 9, 16)
    for x in (u, w):
        assert abs(x.mean() - 0.5) < 0.01 and abs(x.var() * 12 - 1) < 0.02
    assert abs(np.corrcoef(u, w)[0, 1]) < 0.02
    assert abs(np.corrcoef(u, oracle.dither(np.arange(1 << 16), 5, 10, 0))[0, 1]) < 0.02
    assert abs(np.corrcoef(u, oracle.dither(np.arange(1 << 16), 6, 9, 0))[0, 1]) < 0.02
    big = np.array([0, 1 << 34, 1 << 35])
    assert len(set(oracle.dither(big, 5, 9, 0))) == 3


def test_oracle_grad_norm():
    r = np.random.default_rng(1)
    gs = [r.standard_normal(1000).astype(np.float32), r.standard_normal(7)]
    norm, factor = oracle.grad_norm(gs, 1.0)
    assert abs(norm - np.linalg.norm(np.concatenate(gs))) <= 1e-13 * norm
    assert factor == np.float32(1.0 / norm)
    assert oracle.grad_norm(gs, 1e9) == (norm, np.float32(1.0))
    assert oracle.grad_norm([], 1.0) == (0.0, np.float32(1.0))
    n, f = oracle.grad_norm([np.array([1.0, np.inf])], 1.0)
    assert n == math.inf and np.isnan(f)
    n, f = oracle.grad_norm([np.array([np.nan, np.inf])], 1.0)
    assert np.isnan(n) and np.isnan(f)


def test_moments_helper_matches_oracle():
    import torch
    r = np.random.default_rng(8)
    n = 100
    codes = r.integers(0, 256, n).astype(np.uint8)
    e = np.array([0, 17, 255, 200], np.uint8)
    t = (torch.from_numpy(codes).view(torch.float8_e4m3fn), torch.from_numpy(e)) * 2
    m, v = ms.adamw8_moments(t)
    ref = oracle.moment_values(codes, e).astype(np.float32)
    assert np.array_equal(m.numpy(), ref, equal_nan=True) and np.array_equal(v.numpy(), ref, equal_nan=True)
