"""The norm's rows have d values each: shapes that merely hold as many values are refused. GPU
tensors without a GPU (fake ones, whose null address the library refuses) stand in for real
ones."""

import ctypes

import pytest
import torch

try:
    from contextual_activation_sparsity_amd import binding as B
except ImportError:  # library not built
    B = None

pytestmark = [pytest.mark.skipif(B is None, reason="libsparse_ffn.so not built"), pytest.mark.filterwarnings("ignore")]


@pytest.mark.parametrize("shape", [(8, 32), (2, 128), (256,), (64, 4), ()])
@pytest.mark.parametrize("which", ["h", "y", "gate"])
def test_norm_rows_of_another_length_are_refused(which, shape):
    from torch._subclasses.fake_tensor import FakeTensorMode

    n = B.sfn_norm(64, 1, 1e-5, 1.0, 0x100000, 0x100000)
    with FakeTensorMode():
        row = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        a = dict(h=row(4, 64), y=row(4, 64), h_out=None, x_out=row(4, 64), gate=None)
        assert B._args.norm(ctypes.addressof(n), *a.values(), 0) == B.SFN_EINVAL  # fits; then the null addresses
        a[which] = row(*shape)
        with pytest.raises(ValueError, match=rf"{which} must be \[T, 64\]"):
            B._args.norm(ctypes.addressof(n), *a.values(), 0)
