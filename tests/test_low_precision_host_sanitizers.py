"""The host code of root-mean-square norm, 4-bit matrices and their product under
AddressSanitizer and UndefinedBehaviorSanitizer (see test_host_sanitizers.py), on
the CPU."""
import os
import subprocess
import sys

import pytest

from test_host_sanitizers import ROOT, _stale


def test_low_precision_abi_suite_under_host_asan_and_ubsan():
    from adamw_optimizer_step_amd import build as B
    if not os.path.exists(B.HIPCC):
        pytest.skip("hipcc not available")
    if _stale(B.SAN_LIB):
        B.build_host_sanitized(verbose=False)
    env = dict(os.environ, LD_PRELOAD=B.asan_runtime(), MA_LIBRARY=B.SAN_LIB,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_low_precision_abi.py")], cwd=ROOT, env=env, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-3000:])
    assert "passed" in r.stdout
