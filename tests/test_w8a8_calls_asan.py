"""The 8-bit operators' further host tests (overlaps, sums, plans, workspaces) under AddressSanitizer and UndefinedBehaviorSanitizer, in
a child process."""
import os
import subprocess
import sys

import pytest

from test_host_asan import ROOT, _runtime


def test_w8a8_call_tests_pass_under_sanitizers():
    asan, ubsan = _runtime("libasan.so"), _runtime("libubsan.so")
    if not asan or not ubsan:
        pytest.skip("gcc sanitizer runtimes not installed")
    sys.path.insert(0, os.path.join(ROOT, "weight_only_quantized_qgemm_amd"))
    try:
        import _build_asan
    finally:
        sys.path.pop(0)
    env = dict(os.environ, LD_PRELOAD=f"{asan}:{ubsan}", QGEMM_LIB_PATH=_build_asan.build_asan(),
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_w8a8_calls.py", "-q", "-x", "-s", "-p",
                        "no:cacheprovider"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "runtime error" not in out and "AddressSanitizer" not in out and " passed" in out, out[-4000:]
