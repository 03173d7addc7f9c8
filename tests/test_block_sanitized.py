"""The size queries of the operators around the long convolution under
AddressSanitizer and UndefinedBehaviorSanitizer (tests/abi_check_block.c), on the CPU."""
import os
import subprocess

import pytest

from subquadratic_sequence_amd import build as hybuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_size_queries_under_sanitizers():
    if not os.path.exists(os.path.join(ROOT, "subquadratic_sequence_amd", "libhyena.so")):
        pytest.skip("libhyena.so not built")
    exe = hybuild.build_abi_check(name="abi_check_block")
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "all expectations hold" in r.stdout and "runtime error" not in r.stderr
