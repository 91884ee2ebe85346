"""The workspace of attention over a shared prefix on the CPU: how large it is, and that no call
needs more than the size query says."""

import pytest

try:
    from contextual_activation_sparsity_amd import binding as B
except ImportError:  # library not built
    B = None

from tests.test_abi_cache8 import FAKE, _kv, _kv8, shared

pytestmark = [pytest.mark.skipif(B is None, reason="libsparse_ffn.so not built"), pytest.mark.filterwarnings("ignore")]

HEADER = 2048
# Rows of parts that split keys take at most: of the requests' own keys 32 rows for each of 3200
# workgroups (128 for each of 256 in tiles), of the prefix's 128 for each of 2048
SPLIT_OWN, SPLIT_PREFIX = 32 * 3200, 128 * 2048


def size(kv, *a):
    lib = B.raw()
    return (lib.kv8_cache_attend_shared_workspace_size if isinstance(kv, B.sfn_kv8) else lib.kv_cache_attend_shared_workspace_size)(kv, *a)


@pytest.mark.parametrize("e8", [False, True])
@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("R,T,max_new", [(48, 2095, 2048), (200, 4000, 3000), (64, 64, 4096), (1000, 4096, 262144), (1, 5, 9), (7, 300, 1)])
def test_parts_are_of_the_tokens_and_not_of_the_bounds(R, T, max_new, dtype, e8):
    """A token has parts of both sets of keys, 4 dh + 8 bytes for each of its heads, or as many as its
    keys have splits; a bound on the requests' tokens that is far from the truth adds nothing."""
    kv = (_kv8 if e8 else _kv)(dtype=dtype)
    h_q, own, prefix = 32, 3000, 8000
    rows = T * h_q
    most = (4 * 128 + 8) * (max(rows, SPLIT_OWN) + max(rows, SPLIT_PREFIX)) + HEADER + 4 * 256
    need = size(kv, R, T, h_q, max_new, prefix, own)
    assert 0 < need <= most
    # and the call itself asks for no more (its next check is the workspace's alignment), nor do smaller ones
    for r, t, n in {(R, T, max_new), (R, max(1, T // 3), max_new), (max(1, R // 2), T, max_new), (R, T, max(1, max_new // 7)), (1, T, T), (R, T, 1)}:
        if r <= R and n <= max_new:
            assert shared(kv, R=r, T=t, max_new=n, max_shared=prefix, max_own=own, max_pages=9999, prefix_pages=9999, ws=FAKE + 16, ws_bytes=need) == B.SFN_EALIGN


@pytest.mark.parametrize("e8", [False, True])
@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("R,max_new", [(4, 1), (3, 16), (1, 1)])
def test_a_group_of_few_tokens_in_a_large_step(R, max_new, dtype, e8):
    """Other tokens of the step, of other calls' requests, change nothing about a group's work: the
    division of the prefix and its parts are those of a step with this group alone."""
    kv = (_kv8 if e8 else _kv)(dtype=dtype)
    need = size(kv, R, R * max_new, 32, max_new, 60000, 1000)
    assert size(kv, R, 2048, 32, max_new, 60000, 1000) == size(kv, R, 262144, 32, max_new, 60000, 1000) == need > 0
    few = dict(R=R, max_new=max_new, max_shared=60000, max_own=1000, max_pages=9999, prefix_pages=9999)

    # what the call itself asks for
    def asks(T):
        lo, hi = HEADER, need
        while lo < hi:
            mid = (lo + hi) // 2
            lo, hi = (lo, mid) if shared(kv, T=T, ws_bytes=mid, ws=FAKE + 16, **few) == B.SFN_EALIGN else (mid + 1, hi)
        return lo

    assert asks(R * max_new) == asks(2048)
