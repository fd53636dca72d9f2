"""The dense side's argument checks under AddressSanitizer and UndefinedBehaviorSanitizer: the CPU
tests of its C ABI run against the sanitized host build in a child process, as the host runtime's
do; a report aborts the child."""
import os
import subprocess
import sys

import pytest

pytest.importorskip("torch")

from tests.test_sanitized_host_cpu import ROOT, _runtime  # noqa: E402


def test_dense_checks_under_asan_and_ubsan():
    asan = _runtime("libasan.so")
    if asan is None:
        pytest.skip("g++ has no AddressSanitizer runtime here")
    from ad_recommendation_amd import build as B
    env = dict(os.environ, MI355EMB_LIB=B.build_sanitized(), LD_PRELOAD=asan,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                        "tests/test_dense_cpu.py"], cwd=ROOT, env=env, stdout=subprocess.PIPE,
                       stderr=subprocess.STDOUT, text=True, timeout=600)
    assert r.returncode == 0 and " passed" in r.stdout, "\n".join(r.stdout.splitlines()[-30:])
