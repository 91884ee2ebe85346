"""What the compiled tensor checks do with tensors that torch itself refuses to give an
address of (a batched tensor inside ``torch.vmap`` has no storage): torch's error is raised,
as the checks in Python raise it. In a child process, which an exception that left the
module as a C++ one would end."""

import os
import subprocess
import sys

import pytest

try:
    from contextual_activation_sparsity_amd import binding as B
except ImportError:  # library not built
    B = None

pytestmark = pytest.mark.skipif(B is None, reason="libsparse_ffn.so not built")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import ctypes, torch
from torch._subclasses.fake_tensor import FakeTensorMode
from contextual_activation_sparsity_amd import binding as B

kv = B.sfn_kv(8, 16, 2, 64, 1, 0, 0x100000, 0x100000)
nm = B.sfn_norm(64, 1, 1e-5, 1.0, 0x100000, 0x100000)
kv_at, nm_at = ctypes.addressof(kv), ctypes.addressof(nm)

def refused(call, *args):
    try:
        call(*args)
    except RuntimeError as e:
        assert "storage" in str(e), e
        print("refused", flush=True)

def each(rows, ints):
    refused(B._ptr, rows, "x")  # the checks in Python
    refused(B._args.plan, kv_at, *[ints] * 12, 0)
    refused(B._args.append, kv_at, rows, rows, ints, None, None, None, None, 0)
    refused(B._args.attend, kv_at, rows, ints, ints, ints, rows, rows, 1, 1, 1.0, 0, 0)
    refused(B._args.norm, nm_at, rows, None, None, rows, None, 0)
    return rows

with FakeTensorMode():  # GPU tensors without a GPU
    torch.vmap(each)(torch.empty(3, 4, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 4, dtype=torch.int32, device="cuda"))
"""


def test_torch_errors_are_raised():
    res = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, (res.returncode, res.stderr[-2000:])
    assert res.stdout.split() == ["refused"] * 5
