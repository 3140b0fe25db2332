"""Which kernels the host code launches, and on what memory: the library's objects with a HIP runtime that only records
(tests/hip_recorder.c)."""

import ctypes
import os
import subprocess

import pytest

import muon_step_amd as ms
from test_blocks_router_cpu import BASE, block, router
from test_sanitize_cpu import BUILD, ROOT


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    from muon_step_amd import build as b
    objs = [os.path.join(BUILD, src + ".o") for src in b.SOURCES]
    if not all(os.path.exists(o) for o in objs):
        pytest.fail("objects are not built (run __graft_entry__.build())")
    tmp = tmp_path_factory.mktemp("recorder")
    stub, out = str(tmp / "recorder.o"), str(tmp / "librecorded.so")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-O1", "-fPIC", "-c", os.path.join(ROOT, "tests", "hip_recorder.c"),
                    "-o", stub], check=True)
    # names are bound within the library, whatever HIP runtime the process has
    subprocess.run(["g++", "-shared", "-Wl,-Bsymbolic", "-Wl,-z,defs", *objs, stub, "-o", out], check=True)
    lib = ctypes.CDLL(out)
    lib.recorder_name.restype = ctypes.c_char_p
    lib.recorder_arg.restype = ctypes.c_uint64
    lib.muon_last_error.restype = ctypes.c_char_p
    return lib


class Recorded:
    def __init__(self, lib, cap=0):
        self.lib, self.handle = lib, ctypes.c_void_p()
        lib.recorder_capture(0)
        lib.recorder_refuse_memory(0)
        assert lib.muon_create(ctypes.byref(self.handle), 0, ctypes.c_size_t(cap)) == ms.MUON_OK

    def calls(self, what):
        """The status of a call, and its launches: name, workgroups, the first two arguments where they are kept."""
        self.lib.recorder_reset()
        st = what()
        return st, [(self.lib.recorder_name(i).decode(), self.lib.recorder_blocks(i), self.lib.recorder_arg(i, 0),
                     self.lib.recorder_arg(i, 1)) for i in range(self.lib.recorder_count())]

    def balance(self, *routers):
        arr = (ms.muon_router * len(routers))(*routers)
        hp = ms.balance_hparams(1e-3)
        return self.calls(lambda: self.lib.muon_router_balance(self.handle, arr, ctypes.c_int64(len(routers)), ctypes.byref(hp),
                                                               None))

    def blocks(self, coeffs, *mats):
        arr = (ms.muon_block_matrix * len(mats))(*mats)
        hp = ms.make_hparams(coeffs=coeffs)
        return self.calls(lambda: self.lib.muon_blocks_step(self.handle, arr, ctypes.c_int64(len(mats)), ctypes.byref(hp), None))


@pytest.fixture()
def ctx(lib):
    c = Recorded(lib)
    yield c
    lib.muon_destroy(c.handle)


def kinds(calls):
    for c in calls:
        assert "_kernel" in c[0], c
    return [c[0].split("_kernel")[0].split("N_1")[-1].lstrip("0123456789") for c in calls]


def packed(sequences, tokens=9000):
    return router(tokens=tokens, offsets=BASE + (6 << 32), sequences=sequences)


def test_counts_are_cleared_in_other_memory(ctx):
    """Counts lie at zero between calls; where they outgrow their memory, all of the new one is cleared, although it may
    begin where the old one did."""
    st, calls = ctx.balance(packed(2))
    assert st == ms.MUON_OK and kinds(calls) == ["router_clear", "router_count", "router_balance", "router_finish"]
    begin, words = calls[0][2:]
    assert words == 2 * 65
    assert kinds(ctx.balance(packed(1))[1]) == kinds(ctx.balance(packed(2))[1]) == kinds(calls)[1:]
    for sequences in (3, 9, 100):
        st, calls = ctx.balance(packed(sequences))
        assert st == ms.MUON_OK and kinds(calls)[0] == "router_clear"
        assert calls[0][2:] == (begin, sequences * 65), "the recorder gives freed memory out again"
        assert kinds(ctx.balance(packed(sequences))[1])[0] == "router_count"


def test_counts_in_memory_of_a_refused_call(ctx):
    """Memory that could not be had leaves nothing to rely on; the next call clears what it gets."""
    ctx.balance(packed(4))
    ctx.lib.recorder_refuse_memory(1)
    st, calls = ctx.balance(packed(40))
    assert st == ms.MUON_ERR_OUT_OF_MEMORY and not calls
    ctx.lib.recorder_refuse_memory(0)
    st, calls = ctx.balance(packed(2))
    assert st == ms.MUON_OK and calls[0][3] == 2 * 65
    ctx.lib.recorder_capture(1)
    assert ctx.balance(packed(3))[0] == ms.MUON_ERR_UNSUPPORTED
    st, calls = ctx.balance(packed(2))
    ctx.lib.recorder_capture(0)
    assert st == ms.MUON_OK and kinds(calls) == ["router_count", "router_balance", "router_finish"]


def test_many_sequences_are_spread(ctx):
    """The last launch adds up all counts of all sequences: one workgroup for each router and 16384 of them, in whole
    sequences (252 of 65, 63 of 257, 16 of 1024), or more where that would be above 1024 workgroups."""
    for sequences, experts, workgroups in ((1, 64, 1), (252, 64, 1), (253, 64, 2), (4096, 256, 66), (1 << 20, 1023, 1024)):
        one = router(tokens=1 << 20, offsets=BASE + (8 << 32), sequences=sequences, experts=experts, pitch=1024, dlogits_pitch=1024)
        st, calls = ctx.balance(one)
        assert st == ms.MUON_OK and kinds(calls)[-1] == "router_finish" and calls[-1][1] == workgroups, sequences
        few = router(1, tokens=9000, experts=experts, pitch=1024, dlogits_pitch=1024)
        assert ctx.balance(one, few)[1][-1][1] == 2 * workgroups


QUINTIC, CUBIC = (3.4445, -4.7750, 2.0315), (2.0, -1.5, 0.5)


@pytest.mark.parametrize("coeffs, segments", [
    ([], 1), ([CUBIC], 1), ([QUINTIC] * 3, 1), ([QUINTIC] * 4, 2), ([QUINTIC] * 5, 2), ([QUINTIC] * 8 + [CUBIC] * 2, 2),
    ([QUINTIC] * 12, 4), ([QUINTIC] * 8 + [CUBIC], 3), ([CUBIC] * 9, 1), ([CUBIC] * 20, 3)])
def test_passes_of_a_schedule(ctx, coeffs, segments):
    """One Gram pass between two segments; blocks with a side of up to 16 take none."""
    st, calls = ctx.blocks(coeffs, block())
    assert st == ms.MUON_OK
    assert kinds(calls) == ["blocks_momentum"] + ["blocks_chain", "blocks_regram"] * (segments - 1) + ["blocks_chain", "blocks_update"]
    for narrow in (block(block_rows=16), block(rows=16, block_rows=1), block(block_rows=256, block_cols=8)):
        st, calls = ctx.blocks(coeffs, narrow)
        assert st == ms.MUON_OK and kinds(calls) == ["narrow_momentum", "narrow_chain", "blocks_update"]
