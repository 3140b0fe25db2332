"""The argument checks of the mixed-type AdamW steps and the gradient norm under AddressSanitizer and
UndefinedBehaviorSanitizer: runtime.cpp's host code rebuilt with them, driven by adamw_sanitize_driver.c with fake
device pointers.  Needs no GPU."""

import os

import pytest

from test_sanitize_cpu import BUILD, HIPCC, ROOT, SAN, _run


def test_adamw_checks_under_asan_and_ubsan(tmp_path):
    from muon_step_amd import build as b
    objs = [os.path.join(BUILD, src + ".o") for src in b.SOURCES if src != "runtime.cpp"]
    if not all(os.path.exists(o) for o in objs):
        pytest.fail("kernel objects are not built (run __graft_entry__.build())")
    rt, lib, exe = (str(tmp_path / n) for n in ("runtime_san.o", "libmuon_step_san.so", "driver"))
    _run([HIPCC, *b.COMMON, *SAN, "-c", os.path.join(b.CSRC, "runtime.cpp"), "-o", rt])
    _run([HIPCC, "-shared", "-fPIC", f"--offload-arch={b.ARCH}", *SAN, rt, *objs, "-o", lib])
    _run([HIPCC, *SAN, "-x", "c", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
          os.path.join(ROOT, "tests", "adamw_sanitize_driver.c"), "-x", "none", lib, "-o", exe, f"-Wl,-rpath,{tmp_path}"])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    res = _run([exe], env=env, timeout=300)
    assert "sanitized AdamW checks: ok" in res.stdout
    assert "runtime error" not in res.stderr
