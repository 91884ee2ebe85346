"""The binding without its compiled tensor checks (not built, or built for another torch or
Python): the FFN's calls, which do not use them, are there; the paged cache's and the norm's
say what is missing when they are called. In child processes, each with a stand-in for the
module."""

import os
import subprocess
import sys

import pytest
import torch

try:
    from contextual_activation_sparsity_amd import binding as B
except ImportError:  # library not built
    B = None

pytestmark = pytest.mark.skipif(B is None, reason="libsparse_ffn.so not built")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import sys, types
stand_in = types.ModuleType("_torch_args")
{setup}
sys.modules["contextual_activation_sparsity_amd._torch_args"] = stand_in
from contextual_activation_sparsity_amd import binding as B
ffn = B.sfn_ffn(256, 688, 1, 0, 0x100000, 0x100000, 0x100000, None)
assert B.raw().sparse_ffn_workspace_size(ffn, 16) > 0
assert B.raw().kv_cache_attend_workspace_size(B.sfn_kv(9, 16, 2, 64, 1, 0, None, None), 1, 1, 2, 1, 100) > 0
kv = types.SimpleNamespace(addr=0, dh=64)
for call, args in ((B.kv_cache_plan, 12), (B.kv_cache_append, 3), (B.kv_cache_attend, 8), (B.residual_norm, 4)):
    try:
        call(kv, *[None] * args, stream=0)
    except ImportError as e:
        assert {what!r} in str(e) and "contextual_activation_sparsity_amd.build" in str(e), e
        print("refused", flush=True)
"""
BIND = "stand_in.bind = lambda *a: None\n"


@pytest.mark.parametrize("setup,what", [
    ("stand_in = None", "_torch_args"),
    (BIND + "stand_in.TORCH_VERSION, stand_in.PY_VERSION = '1.0.0', '%d.%d' % sys.version_info[:2]", "torch 1.0.0"),
    (BIND + f"stand_in.TORCH_VERSION, stand_in.PY_VERSION = {torch.__version__!r}.split('+')[0], '2.7'", "Python 2.7"),
    ("pass", "_torch_args")], ids=["missing", "torch", "python", "older"])
def test_ffn_calls_without_the_checks(setup, what):
    res = subprocess.run([sys.executable, "-c", CHILD.format(setup=setup, what=what)], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stderr[-2000:]
    assert res.stdout.split() == ["refused"] * 4


def test_built_module_names_what_it_was_built_for():
    assert torch.__version__.startswith(B._args.TORCH_VERSION) and B._args.PY_VERSION == "%d.%d" % sys.version_info[:2]
