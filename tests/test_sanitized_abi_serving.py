"""The paged cache's and the residual norm's host code under AddressSanitizer and
UndefinedBehaviorSanitizer: tests/test_abi_serving.py in a child process on the
host-sanitized build, as tests/test_sanitized_abi.py does for the other calls."""

import os
import subprocess
import sys

import pytest

from tests.test_sanitized_abi import CLANG, ROOT, SAN_LIB, _stale


@pytest.mark.skipif(_stale() is not None, reason=str(_stale()))
def test_serving_abi_under_asan_and_ubsan():
    rt = subprocess.run([CLANG, "-print-file-name=libclang_rt.asan-x86_64.so"], capture_output=True, text=True,
                        check=True).stdout.strip()
    env = dict(os.environ, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1", SFN_LIBRARY=SAN_LIB)
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-m", "not gpu",
                          os.path.join("tests", "test_abi_serving.py")], cwd=ROOT, env=env, capture_output=True, text=True,
                         timeout=600)
    out = res.stdout + res.stderr
    assert res.returncode == 0 and "passed" in res.stdout, out[-4000:]
    assert "ERROR: AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
