"""Calls of the mixed-type AdamW steps, the gradient norm and the clip factor that their documentation allows or rules
out, where one was once answered wrongly; needs no GPU."""

import ctypes
import os
import re
import subprocess
import sys

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


def test_load_refuses_another_abi(tmp_path, monkeypatch):
    """A library built from another version of the header lays its structures out differently: it is not loaded."""
    src = tmp_path / "old.c"
    src.write_text("int muon_abi_version(void) { return 4; }\n")
    so = str(tmp_path / "old.so")
    subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", so], check=True)
    monkeypatch.setattr(ms, "_lib", None)
    with pytest.raises(ImportError, match=r"ABI version 4.*needs 5"):
        ms.load(so)
    assert ms._lib is None


def test_abi_version_is_the_headers():
    """The version that load() asks for is the one of the header that the structures mirror."""
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "muon_step.h")
    m = re.search(r"#define MUON_STEP_ABI_VERSION (\d+)", open(header).read())
    assert ms.MUON_STEP_ABI_VERSION == int(m.group(1))


def _status(fn, ts, *args):
    arr = (type(ts[0]) * len(ts))(*ts)
    buf = ctypes.create_string_buffer(512)
    return fn(arr, len(ts), *args, buf, 512), buf.value.decode()


@pytest.mark.parametrize("kind", [ms.muon_adamw_mixed_tensor, ms.muon_adamw8_tensor])
@pytest.mark.parametrize("dtype", [ms.MUON_F32, ms.MUON_BF16])
def test_pointers_of_an_empty_tensor_are_not_looked_at(kind, dtype):
    """Not the master copy's either, whatever the weights' type; a tensor with elements is refused as before."""
    lib = ms.load()
    fn = lib.muon_check_adamw_mixed_args if kind is ms.muon_adamw_mixed_tensor else lib.muon_check_adamw8_args
    hp = ms.adamw_hparams()
    t = kind(param=3, master=5, grad=7, exp_avg=9, exp_avg_sq=11, numel=0, param_dtype=dtype, grad_dtype=ms.MUON_F32)
    assert _status(fn, [t], ctypes.byref(hp), None) == (ms.MUON_OK, "")
    t.numel = 1
    assert _status(fn, [t], ctypes.byref(hp), None)[0] == ms.MUON_ERR_INVALID_ARGUMENT


def test_overlap_messages_name_the_factor():
    """The clip factor belongs to no matrix or tensor: the message names it without a number."""
    lib = ms.load()
    base = 1 << 40
    mats = [ms.muon_matrix(base + (i << 36), base + (i << 36) + (1 << 30), base + (i << 36) + (2 << 30), None, 64, 128,
                           ms.MUON_BF16, ms.MUON_BF16) for i in range(2)]
    hp = ms.make_hparams()
    for at, what in ((mats[1].momentum + 16, "matrix 1 momentum"), (mats[1].param, "matrix 1 param"),
                     (mats[0].momentum + 4 * 64 * 128 - 4, "matrix 0 momentum")):
        hp.grad_factor = at
        st, msg = _status(lib.muon_check_step_args, mats, ctypes.byref(hp))
        assert st == ms.MUON_ERR_INVALID_ARGUMENT
        assert msg in (f"memory of {what} overlaps grad_factor", f"memory of grad_factor overlaps {what}")
    mats[1].param = mats[0].momentum
    hp.grad_factor = None
    st, msg = _status(lib.muon_check_step_args, mats, ctypes.byref(hp))
    assert st == ms.MUON_ERR_INVALID_ARGUMENT
    assert sorted(msg[len("memory of "):].split(" overlaps ")) == ["matrix 0 momentum", "matrix 1 param"]

    def tensor(kind, i):
        names = [f for f, t in kind._fields_ if t is ctypes.c_void_p and f != "master"]
        at = {f: base + (i << 36) + (k << 20) for k, f in enumerate(names)}
        return kind(**at, numel=1000, param_dtype=ms.MUON_F32, grad_dtype=ms.MUON_F32)

    for kind, fn in ((ms.muon_adamw_mixed_tensor, lib.muon_check_adamw_mixed_args),
                     (ms.muon_adamw8_tensor, lib.muon_check_adamw8_args)):
        ts = [tensor(kind, i) for i in range(3)]
        st, msg = _status(fn, ts, ctypes.byref(ms.adamw_hparams()), ts[2].exp_avg_sq + 4)
        assert st == ms.MUON_ERR_INVALID_ARGUMENT
        assert msg in ("memory of tensor 2 exp_avg_sq overlaps grad_factor",
                       "memory of grad_factor overlaps tensor 2 exp_avg_sq")


@pytest.mark.parametrize("args", [["--workload", "moe16b", "--clip-norm", "0"],
                                  ["--workload", "moe16b", "--clip-norm", "-1"],
                                  ["--workload", "moe16b", "--clip-norm", "nan"],
                                  ["--clip-norm", "1"], ["--adamw8"],
                                  ["--workload", "dense_block_bf16", "--clip-norm", "1"]])
def test_bench_refuses_options_that_would_do_nothing(args):
    """A norm that the library refuses, and options of another workload, end the run before it starts."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, os.path.join(root, "bench.py"), *args], capture_output=True, text=True,
                         timeout=100)
    assert res.returncode == 2 and res.stdout == ""
    assert "--clip-norm" in res.stderr.splitlines()[-1] or "--adamw8" in res.stderr.splitlines()[-1]


def test_oracle_8_bit_weights_are_those_of_the_32_bit_step():
    """From the same moments the weights of the two steps differ by fp32 roundings alone, at second moments up to
    fp32's largest value.  In units of 2^-24: the 32-bit step rounds v / (1 - b2^t) (halved by the root), the root, the
    sum with eps, two quotients, the product with lr and three constants: at most 9 of the update; the decay's constant
    and product and the difference: at most 3 of the larger weight."""
    rng = np.random.default_rng(22)
    n = 64 * 32
    for step in (1, 3, 1000):
        e = np.repeat(np.linspace(20, 240, 64).astype(np.uint8), 1)          # v from 2^-116 to past 2^120
        state = (rng.integers(0, 127, n).astype(np.uint8), ((e.astype(int) + 127) // 2).astype(np.uint8),
                 rng.integers(8, 127, n).astype(np.uint8), e)
        m, v = (oracle.moment_values(c, s).astype(np.float32) for c, s in (state[:2], state[2:]))
        p, g = rng.standard_normal(n).astype(np.float32), np.zeros(n, np.float32)
        args = (0.02, 0.9, 0.95, 1e-8, 0.1, step)
        with np.errstate(over="ignore"):
            p32, m32, v32 = oracle.adamw_step_f32(p, g, m, v, *args)
            p8, update, _ = oracle.adamw8_step(p, g, state, *args)
        assert np.isfinite(v32).all() and v32.max() > 2.0 ** 120
        assert (np.abs(p8 - p32) <= 2.0 ** -24 * (9 * np.abs(update) + 3 * np.maximum(np.abs(p), np.abs(p32)))).all()


def test_no_exception_leaves_the_checks():
    """A count that no host memory could list is an error, not the end of the process."""
    code = """if True:
        import ctypes, muon_step_amd as ms
        lib, buf = ms.load(), ctypes.create_string_buffer(100)
        mats, need = (ms.muon_matrix * 1)(), ctypes.c_size_t()
        for count in (1 << 62, 1 << 60, (1 << 63) - 1):
            hp = ctypes.byref(ms.make_hparams())
            print(lib.muon_check_step_args(mats, count, hp, buf, 100), buf.value.decode())
            print(lib.muon_check_step_args(mats, count, hp, None, 0))
            print(lib.muon_workspace_bytes(mats, count, hp, ctypes.byref(need)))
        """
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=100)
    assert res.returncode == 0, res.stderr
    out = ms.MUON_ERR_OUT_OF_MEMORY
    assert res.stdout.splitlines() == [f"{out} out of host memory", f"{out}", f"{out}"] * 3


def test_slow_second_moment_over_many_steps():
    """A second moment at b2 = 0.999 over 2000 steps of constant gradients: unbiased, and its noise stays within what
    the rounding's variance gives.  A step moves a code c by d <= (1 - b2) c at most once it is settled, and rounds with
    variance at most d x gap <= (1 - b2) c^2 / 8 (the gap is c / 8 at most); the sum over the steps, each weakened by
    b2 a step, is at most 1 / (1 - b2^2) of that: c^2 / 16, a standard deviation of a quarter.  4096 elements are 1024
    independent groups of four: their mean is within 5 x 1/4 / 32 = 4% of the exact one, and their deviation's estimate
    within 5 / sqrt(2 x 1024) = 11% of the true one."""
    n, steps, b2 = 4096, 2000, 0.999
    rng = np.random.default_rng(23)
    g = np.exp2(rng.uniform(-1, 1, n)).astype(np.float32)
    k = oracle.adamw_scalars_f32(0.02, 0.9, b2, 1e-8, 0.1, 1)
    codes, scale = np.zeros(n, np.uint8), np.zeros(n // 32, np.uint8)
    index = np.arange(n)
    for step in range(1, steps + 1):
        v = oracle.moment_values(codes, scale).astype(np.float32)
        v = (k["beta2"] * v) + ((k["one_minus_beta2"] * g) * g)
        codes, scale = oracle.quantise(v, True, index, 99, step, 16)
    ratio = oracle.moment_values(codes, scale) / ((1 - b2 ** steps) * g.astype(np.float64) ** 2)
    assert abs(ratio.mean() - 1) <= 0.04
    assert ratio.std() <= 0.25 * 1.11


def test_words_of_the_two_moments():
    """What the rounding's words share, as the format is defined: a group of four elements has one word, turned by a
    byte for each, and an element's second moment takes the turn of the first moment of the element two further on."""
    i = np.arange(64)
    first, second = oracle.dither(i, 7, 3, 0), oracle.dither(i, 7, 3, 16)
    assert np.array_equal(second, first[i // 4 * 4 + (i + 2) % 4])
