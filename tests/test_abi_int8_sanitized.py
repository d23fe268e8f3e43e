"""The int8 and scored-router ABI checks (tests/test_abi_int8.py) against the library
whose host code runs under AddressSanitizer and UndefinedBehaviorSanitizer, as
tests/test_abi_sanitized.py does for the others."""

import os
import subprocess
import sys

import pytest

from test_abi_sanitized import ROOT, _hipcc, _stale


def test_int8_abi_checks_pass_under_asan_and_ubsan():
    hipcc = _hipcc()
    if hipcc is None:
        pytest.skip("hipcc not available")
    from block_diffusion_lm_tq4_amd import build as B
    lib = B.SANITIZED_LIB
    if _stale(lib):
        B.build_sanitized()
    runtime = subprocess.run([hipcc, "-print-file-name=libclang_rt.asan-x86_64.so"],
                             capture_output=True, text=True).stdout.strip()
    assert os.path.exists(runtime), runtime
    env = dict(os.environ)
    env.update(TQ4_LIBRARY=lib, LD_PRELOAD=runtime,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                          os.path.join(ROOT, "tests", "test_abi_int8.py")],
                         cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = res.stdout + res.stderr
    assert res.returncode == 0, out[-4000:]
    assert "passed" in out and "ERROR: AddressSanitizer" not in out and "runtime error" not in out
