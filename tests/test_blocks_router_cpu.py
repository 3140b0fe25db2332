"""muon_blocks_step, muon_router_balance and muon_router_bias_step without a GPU: structure layouts, what the checks and the
tensor functions refuse and allow, the checks under sanitizers."""

import ctypes
import os
import re
import subprocess
import sys

import pytest

import muon_step_amd as ms
from test_sanitize_cpu import BUILD, HIPCC, ROOT, SAN, _run

STRUCTS = [ms.muon_block_matrix, ms.muon_router, ms.muon_balance_hparams, ms.muon_router_bias]
BASE = 1 << 40


def test_structures_match_the_header(tmp_path):
    body = "".join(f'printf("{k.__name__} %zu\\n", sizeof({k.__name__}));' +
                   "".join(f'printf("{k.__name__}.{f[0]} %zu\\n", offsetof({k.__name__}, {f[0]}));' for f in k._fields_)
                   for k in STRUCTS)
    src = tmp_path / "layout.c"
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"muon_step.h\"\nint main(void) { " + body + " return 0; }\n")
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    got = dict(line.split() for line in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines())
    for k in STRUCTS:
        assert int(got[k.__name__]) == ctypes.sizeof(k)
        for f in k._fields_:
            assert int(got[f"{k.__name__}.{f[0]}"]) == getattr(k, f[0]).offset, f


def test_limits_are_the_headers():
    header = open(os.path.join(ROOT, "include", "muon_step.h")).read()
    assert ms.MUON_BLOCK_SIDE == int(re.search(r"#define MUON_BLOCK_SIDE (\d+)", header).group(1))


def block(at=0, **kw):
    f = dict(param=BASE + (at << 36), grad=BASE + (at << 36) + (1 << 32), momentum=BASE + (at << 36) + (2 << 32), ns_out=None,
             rows=256, cols=1000, block_rows=64, block_cols=1000, param_pitch=1000, grad_pitch=1000, momentum_pitch=1000,
             ns_out_pitch=0, param_dtype=ms.MUON_BF16, grad_dtype=ms.MUON_BF16)
    f.update(kw)
    return ms.muon_block_matrix(**f)


def check_blocks(items, hp=None):
    msg = ctypes.create_string_buffer(300)
    arr = (ms.muon_block_matrix * max(len(items), 1))(*items)
    hp = ms.make_hparams() if hp is None else hp
    return ms.load().muon_check_blocks_args(arr, len(items), ctypes.byref(hp), msg, 300), msg.value.decode()


@pytest.mark.parametrize("kw", [
    {}, {"block_rows": 1, "block_cols": 1}, {"block_rows": 256, "block_cols": 125}, {"rows": 1, "cols": 1, "block_rows": 1,
                                                                                    "block_cols": 1},
    {"param_pitch": 1 << 26, "param": BASE + (1 << 50)}, {"rows": 128, "block_rows": 128, "cols": 1 << 24,
                                                         "block_cols": 1 << 24, "param_pitch": 1 << 24,
                                                         "grad_pitch": 1 << 24, "momentum_pitch": 1 << 24},
    {"ns_out": BASE + (3 << 32), "ns_out_pitch": 1001}, {"param": BASE + 2}, {"param_dtype": ms.MUON_F32}])
def test_blocks_that_are_taken(kw):
    assert check_blocks([block(**kw)]) == (ms.MUON_OK, "")


@pytest.mark.parametrize("kw, what", [
    ({"rows": 0}, "matrix 0"), ({"cols": -1}, "matrix 0"), ({"block_rows": 0}, "do not divide"),
    ({"block_rows": 48}, "do not divide"), ({"block_cols": 999}, "do not divide"),
    ({"param_pitch": 999}, "param rows"), ({"grad_pitch": 0}, "grad rows"), ({"momentum_pitch": (1 << 26) + 1}, "momentum rows"),
    ({"ns_out": BASE + (3 << 32)}, "ns_out rows"), ({"param": None}, "param is NULL"), ({"momentum": BASE + 2}, "momentum"),
    ({"grad": BASE + (1 << 32) + 1}, "grad"), ({"param_dtype": 7}, "unknown dtype"), ({"grad_dtype": -1}, "unknown dtype"),
    ({"grad": BASE}, "overlaps"), ({"ns_out": BASE + (2 << 32) + 4, "ns_out_pitch": 1000}, "overlaps"),
    ({"momentum": BASE + 1000 * 2}, "overlaps")])
def test_blocks_that_are_refused(kw, what):
    st, msg = check_blocks([block(**kw)])
    assert st == ms.MUON_ERR_INVALID_ARGUMENT and what in msg, (st, msg)


def test_blocks_unsupported():
    assert check_blocks([block(block_rows=256)])[0] == ms.MUON_ERR_UNSUPPORTED
    wide = dict(rows=1, cols=1 << 25, block_rows=1, block_cols=1 << 25, param_pitch=1 << 25, grad_pitch=1 << 25,
                momentum_pitch=1 << 25)
    assert check_blocks([block(**wide)])[0] == ms.MUON_ERR_UNSUPPORTED
    assert check_blocks([block()], ms.make_hparams(ns_precision=ms.MUON_NS_F32))[0] == ms.MUON_ERR_UNSUPPORTED
    for coeffs in ([(5.0, 0.0, 0.0)] * 3, [(3.4445, 4.0, 2.0315)] * 4, [(1.0, 100.0, 0.0)]):
        assert check_blocks([block()], ms.make_hparams(coeffs=coeffs))[0] == ms.MUON_ERR_UNSUPPORTED, coeffs
    for name in ("deepseekv4", "quintic"):
        assert check_blocks([block()], ms.make_hparams(coeffs=ms.schedule(name)))[0] == ms.MUON_OK


def test_blocks_side_by_side_in_one_buffer():
    """Two slices of the columns of one buffer interleave; one element further they meet; another pitch is refused."""
    pair = lambda shift, pitch=4000: [  # noqa: E731
        block(cols=1000, param_pitch=4000), block(1, cols=1000, param=BASE + 2 * shift, param_pitch=pitch)]
    assert check_blocks(pair(1000))[0] == ms.MUON_OK
    assert check_blocks(pair(2000))[0] == ms.MUON_OK
    assert check_blocks(pair(999))[0] == ms.MUON_ERR_INVALID_ARGUMENT
    assert check_blocks(pair(3001))[0] == ms.MUON_ERR_INVALID_ARGUMENT  # its rows reach into the next of the first
    assert check_blocks(pair(1000, 4001))[0] == ms.MUON_ERR_INVALID_ARGUMENT
    assert check_blocks([block(), block()])[0] == ms.MUON_ERR_INVALID_ARGUMENT
    hp = ms.make_hparams()
    hp.grad_factor = BASE + 64
    assert check_blocks([block()], hp)[0] == ms.MUON_ERR_INVALID_ARGUMENT
    hp.grad_factor = BASE + (1 << 32)  # a read one may lie in a gradient
    assert check_blocks([block()], hp)[0] == ms.MUON_OK


def router(at=0, **kw):
    base = BASE + (at << 36)
    f = dict(logits=base, dlogits=base + (1 << 32), chosen=base + (2 << 32), offsets=None, mask=None, counts=base + (3 << 32),
             loss=base + (4 << 32), tokens=1000, pitch=64, dlogits_pitch=64, experts=64, top_k=6, sequences=1,
             dtype=ms.MUON_F32, chosen_bits=64, reserved=0)
    f.update(kw)
    return ms.muon_router(**f)


def check_router(items, hp=None):
    msg = ctypes.create_string_buffer(300)
    arr = (ms.muon_router * max(len(items), 1))(*items)
    hp = ms.balance_hparams(1e-3) if hp is None else hp
    return ms.load().muon_check_router_balance_args(arr, len(items), ctypes.byref(hp), msg, 300), msg.value.decode()


@pytest.mark.parametrize("kw", [
    {}, {"dlogits": None, "dlogits_pitch": 0}, {"experts": 1, "top_k": 1}, {"experts": 1024, "pitch": 1024, "dlogits_pitch": 2048},
    {"mask": BASE + (5 << 32)}, {"offsets": BASE + (6 << 32), "sequences": 5}, {"chosen_bits": 32}, {"top_k": 64},
    {"tokens": 0, "logits": None, "dlogits": None, "chosen": None, "pitch": 0}, {"dtype": ms.MUON_BF16, "logits": BASE + 2},
    {"tokens": 1 << 30, "top_k": 1, "chosen_bits": 32, "experts": 1, "pitch": 1, "dlogits_pitch": 1}])
def test_routers_that_are_taken(kw):
    assert check_router([router(**kw)]) == (ms.MUON_OK, "")


@pytest.mark.parametrize("kw, what", [
    ({"tokens": -1}, "out of range"), ({"tokens": (1 << 30) + 1, "top_k": 1}, "out of range"), ({"experts": 0}, "out of range"),
    ({"experts": 1025, "pitch": 2000}, "out of range"), ({"top_k": 0}, "out of range"), ({"top_k": 65}, "out of range"),
    ({"tokens": 1 << 30, "top_k": 4}, "out of range"), ({"dtype": 3}, "unknown"), ({"chosen_bits": 16}, "unknown"),
    ({"sequences": 0}, "sequences"), ({"sequences": 2}, "without offsets"),
    ({"sequences": (1 << 30) + 1, "offsets": BASE + (6 << 32)}, "sequences"), ({"pitch": 63}, "logits rows"),
    ({"dlogits_pitch": 63}, "dlogits rows"), ({"logits": None}, "logits is NULL"), ({"counts": None}, "counts is NULL"),
    ({"loss": BASE + 2}, "loss"), ({"chosen": BASE + (2 << 32) + 4}, "chosen"), ({"offsets": BASE + 2, "sequences": 2}, "offsets"),
    ({"dlogits": BASE + 64 * 4 * 999 + 4 * 63}, "overlaps"), ({"loss": BASE + (3 << 32)}, "overlaps"),
    ({"counts": BASE + (2 << 32)}, "overlaps"), ({"mask": BASE + (1 << 32) + 5}, "overlaps")])
def test_routers_that_are_refused(kw, what):
    st, msg = check_router([router(**kw)])
    assert st == ms.MUON_ERR_INVALID_ARGUMENT and what in msg, (st, msg)


def test_balance_hparams_that_are_refused():
    for field, value in (("coef", float("nan")), ("coef", float("inf")), ("score", 2), ("accumulate", 2), ("grad_scale", 6),
                         ("grad_scale", BASE + (1 << 32) + 64)):
        hp = ms.balance_hparams(1e-3)
        setattr(hp, field, value)
        assert check_router([router()], hp)[0] == ms.MUON_ERR_INVALID_ARGUMENT, field
    assert check_router([router(), router(1, loss=BASE + (4 << 32))])[0] == ms.MUON_ERR_INVALID_ARGUMENT
    shared = router(1, logits=BASE, chosen=BASE + (2 << 32))  # inputs may be shared
    assert check_router([router(), shared])[0] == ms.MUON_OK


def check_bias(items, rate=1e-3):
    msg = ctypes.create_string_buffer(300)
    arr = (ms.muon_router_bias * max(len(items), 1))(*items)
    return ms.load().muon_check_router_bias_args(arr, len(items), rate, msg, 300)


def test_biases():
    one = lambda **kw: ms.muon_router_bias(**dict(dict(bias=BASE, counts=BASE + 4096, experts=64), **kw))  # noqa: E731
    bad = ms.MUON_ERR_INVALID_ARGUMENT
    assert check_bias([one()]) == ms.MUON_OK == check_bias([]) == check_bias([one(), one(bias=BASE + 256)])
    assert check_bias([one()], float("nan")) == bad == check_bias([one()], 1e39)
    for kw in ({"bias": None}, {"counts": None}, {"experts": 0}, {"experts": (1 << 20) + 1}, {"bias": BASE + 1},
               {"counts": BASE + 4100}, {"counts": BASE + 248}):
        assert check_bias([one(**kw)]) == bad, kw
    assert check_bias([one(), one(bias=BASE + 252)]) == bad


def test_null_lists_and_counts():
    lib, msg = ms.load(), ctypes.create_string_buffer(300)
    hp, bh = ms.make_hparams(), ms.balance_hparams(1.0)
    bad = ms.MUON_ERR_INVALID_ARGUMENT
    assert lib.muon_check_blocks_args(None, 0, ctypes.byref(hp), msg, 300) == ms.MUON_OK
    assert lib.muon_check_router_balance_args(None, 0, ctypes.byref(bh), msg, 300) == ms.MUON_OK
    assert lib.muon_check_router_bias_args(None, 0, 1.0, msg, 300) == ms.MUON_OK
    for count in (1, -1):
        assert lib.muon_check_blocks_args(None, count, ctypes.byref(hp), msg, 300) == bad
        assert lib.muon_check_router_balance_args(None, count, ctypes.byref(bh), msg, 300) == bad
        assert lib.muon_check_router_bias_args(None, count, 1.0, msg, 300) == bad
    assert lib.muon_check_blocks_args((ms.muon_block_matrix * 1)(), 1, None, None, 0) == bad
    assert lib.muon_check_router_balance_args((ms.muon_router * 1)(), 1, None, None, 0) == bad
    assert lib.muon_blocks_step(None, None, 0, ctypes.byref(hp), None) == bad
    assert lib.muon_router_balance(None, None, 0, ctypes.byref(bh), None) == bad
    assert lib.muon_router_bias_step(None, None, 0, 1.0, None) == bad


def test_tensor_functions_refuse():
    """What the descriptors of tensors refuse before any address is taken; CPU tensors come last."""
    import torch
    x = torch.zeros(8, 12)
    for args in ((x[0], x[0], x[0]), (x, x[:4], x), (x.t(), x.t(), x.t()), (x, x, x[:, :0])):
        with pytest.raises(ValueError):
            ms.block_matrix(*args, 4, 12)
    with pytest.raises(ValueError, match="overlap"):
        ms.block_matrix(x[:1].expand(8, 12), x, x, 4, 12)
    for args in ((x, x, x.bfloat16()), (x.half(), x, x)):
        with pytest.raises((TypeError, ValueError)):
            ms.block_matrix(*args, 4, 12)
    with pytest.raises((TypeError, ValueError)):
        ms.block_matrix(x, x, x, 4, 12)
    chosen, counts, loss = torch.zeros(8, 2, dtype=torch.int64), torch.zeros(12, dtype=torch.int64), torch.zeros(1)
    for bad in (dict(logits=x[0]), dict(logits=x.t()), dict(logits=x.half()), dict(chosen=chosen.short()), dict(chosen=chosen[:4]),
                dict(chosen=chosen.t().contiguous().t()), dict(counts=counts.int()), dict(counts=counts[:11]),
                dict(loss=loss.double()), dict(loss=torch.zeros(2)), dict(dlogits=x.bfloat16()), dict(dlogits=x[:4]),
                dict(offsets=torch.zeros(3)), dict(offsets=torch.zeros(1, dtype=torch.int32)), dict(mask=torch.zeros(8)),
                dict(mask=torch.zeros(7, dtype=torch.bool)), dict(dlogits=x[:1].expand(8, 12)), dict()):
        kw = dict(dict(logits=x, chosen=chosen, counts=counts, loss=loss), **bad)
        with pytest.raises((TypeError, ValueError)):
            ms.router(**kw)
    for bad in ((x[0].bfloat16(), counts), (x[0], counts.int()), (x[0], counts[:3]), (x[0, ::2], counts[:6]), (x[0], counts)):
        with pytest.raises((TypeError, ValueError)):
            ms.router_bias(*bad)


def test_checks_under_asan_and_ubsan(tmp_path):
    from muon_step_amd import build as b
    objs = [os.path.join(BUILD, src + ".o") for src in b.SOURCES if src != "runtime.cpp"]
    if not all(os.path.exists(o) for o in objs):
        pytest.fail("kernel objects are not built (run __graft_entry__.build())")
    rt, lib, exe = (str(tmp_path / n) for n in ("runtime_san.o", "libmuon_step_san.so", "driver"))
    _run([HIPCC, *b.COMMON, *SAN, "-c", os.path.join(b.CSRC, "runtime.cpp"), "-o", rt])
    _run([HIPCC, "-shared", "-fPIC", f"--offload-arch={b.ARCH}", *SAN, rt, *objs, "-o", lib])
    _run([HIPCC, *SAN, "-x", "c", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
          os.path.join(ROOT, "tests", "blocks_router_sanitize_driver.c"), "-x", "none", lib, "-o", exe,
          f"-Wl,-rpath,{tmp_path}"])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    res = _run([exe], env=env, timeout=300)
    assert "sanitized block and router checks: ok" in res.stdout
    assert "runtime error" not in res.stderr


@pytest.mark.parametrize("args", [["--head-blocks"], ["--balance"], ["--workload", "dense_block_bf16", "--balance"]])
def test_bench_refuses_options_of_another_workload(args):
    res = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), *args], capture_output=True, text=True, timeout=100)
    assert res.returncode == 2 and res.stdout == ""
    assert "--head-blocks and --balance go with" in res.stderr.splitlines()[-1]


def test_more_blocks_than_a_launch_numbers():
    big = dict(rows=1 << 16, cols=1 << 16, block_rows=1, block_cols=1, param_pitch=1 << 16, grad_pitch=1 << 16,
               momentum_pitch=1 << 16)
    st, msg = check_blocks([block(**big)])
    assert st == ms.MUON_ERR_INVALID_ARGUMENT and "too many blocks" in msg


def test_overlap_against_brute_force():
    """Random layouts in one buffer: what is taken shares no written byte; ranges of one pitch are refused only for one."""
    import random
    rng = random.Random(5)
    taken = refused = 0
    for _ in range(4000):
        items, spans = [], []
        pitches = [rng.choice((8, 8, 8, 12)) for _ in range(2)]
        for i in range(2):
            rows, cols = rng.randint(1, 3), rng.randint(1, 6)
            at = {k: rng.randint(0, 60) for k in ("param", "grad", "momentum")}
            if i or rng.random() < 0.7:  # mostly apart from each other, close to the other weight's
                at = {k: v + 100 * n for n, (k, v) in enumerate(at.items())}
            items.append(block(rows=rows, cols=cols, block_rows=rows, block_cols=cols, param_dtype=ms.MUON_F32,
                               grad_dtype=ms.MUON_F32, **{k: BASE + 4 * v for k, v in at.items()},
                               **{k + "_pitch": pitches[i] for k in at}))
            for k, v in at.items():
                spans.append((k != "grad", pitches[i], {v + r * pitches[i] + c for r in range(rows) for c in range(cols)}))
        pairs = [(a, b) for n, a in enumerate(spans) for b in spans[:n] if a[0] or b[0]]
        shared = any(a[2] & b[2] for a, b in pairs)
        hulls = any(a[1] != b[1] and min(a[2]) <= max(b[2]) and min(b[2]) <= max(a[2]) for a, b in pairs)
        st = check_blocks(items)[0]
        assert st == (ms.MUON_ERR_INVALID_ARGUMENT if shared or hulls else ms.MUON_OK), (items, shared, hulls)
        taken += st == ms.MUON_OK
        refused += st != ms.MUON_OK
    assert taken > 500 and refused > 500, (taken, refused)
