"""The compiled binding lets other Python threads run while the library's function does, as
ctypes does: a launch may wait for room in the queue. In a child process, whose module is
bound to a function of the same kind that sleeps."""

import os
import shutil
import subprocess
import sys

import pytest

try:
    from contextual_activation_sparsity_amd import binding as B
except ImportError:  # library not built
    B = None

pytestmark = [pytest.mark.skipif(B is None, reason="libsparse_ffn.so not built"),
              pytest.mark.skipif(shutil.which("gcc") is None, reason="needs a C compiler")]
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SLEEPER = """
#include <time.h>
static int naps;
int nap(void) { struct timespec t = {0, 400000000}; nanosleep(&t, 0); return ++naps; }
"""

CHILD = """
import ctypes, sys, threading, time
from contextual_activation_sparsity_amd import binding as B
nap = ctypes.cast(ctypes.CDLL(sys.argv[1]).nap, ctypes.c_void_p).value
B._args.bind(*[nap] * 4)
kv = B.sfn_kv(8, 16, 2, 64, 1, 0, 0x100000, 0x100000)
nm = B.sfn_norm(64, 1, 1e-5, 1.0, 0x100000, 0x100000)
calls = [lambda: B._args.plan(ctypes.addressof(kv), *[None] * 12, 0), lambda: B._args.norm(ctypes.addressof(nm), *[None] * 5, 0)]
for n, call in enumerate(calls):
    began, ended, ran = threading.Event(), threading.Event(), []
    def other():
        began.set()
        while not ended.is_set():
            ran.append(time.monotonic())
            time.sleep(0.01)
    t = threading.Thread(target=other)
    t.start()
    began.wait()
    t0 = time.monotonic()
    assert call() == n + 1  # what the function returned
    t1 = time.monotonic()
    ended.set()
    t.join()
    assert t1 - t0 > 0.35
    print(sum(t0 + 0.02 < x < t1 - 0.02 for x in ran), flush=True)
"""


def test_other_threads_run_during_a_call(tmp_path):
    src, lib = tmp_path / "nap.c", tmp_path / "nap.so"
    src.write_text(SLEEPER)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(lib), str(src)], check=True)
    res = subprocess.run([sys.executable, "-c", CHILD, str(lib)], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stderr[-2000:]
    turns = [int(x) for x in res.stdout.split()]
    assert len(turns) == 2 and min(turns) >= 3, turns  # of some 35 in 0.4 s
