"""The attention's workspace query on the CPU: the size for a program's largest bounds is
enough for every call within them. A call checks its workspace's size before its alignment
and both before anything is launched, so a misaligned address tells which it was."""

import random

import pytest

try:
    from contextual_activation_sparsity_amd import binding as B
except ImportError:  # library not built
    B = None

pytestmark = pytest.mark.skipif(B is None, reason="libsparse_ffn.so not built")
FAKE = 0x100000  # never dereferenced: every call below is refused


def enough(kv, h_q, size, R, new, length, window):
    st = B.raw().kv_cache_attend(kv, R, R * new, h_q, FAKE, h_q * kv.dh, FAKE, -(-max(length, 1) // kv.page), FAKE, FAKE, new, length,
                                 0.1, window, FAKE, FAKE + 16, size, None)
    assert st in (B.SFN_EALIGN, B.SFN_EWORKSPACE)
    return st == B.SFN_EALIGN


def size_of(kv, h_q, R, new, length):
    return B.raw().kv_cache_attend_workspace_size(kv, R, R * new, h_q, new, length)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("h_q,h_kv", [(4, 2), (32, 8), (64, 8), (8, 1), (64, 1), (7, 7), (128, 2)])
def test_largest_bounds_cover_smaller_ones(dtype, h_q, h_kv):
    rng = random.Random(h_q * 10 + dtype)
    log = lambda hi: int(round(hi ** rng.random()))  # noqa: E731
    for _ in range(300):
        kv = B.sfn_kv(1000, 16, h_kv, rng.choice([64, 128]), dtype, 0, FAKE, FAKE)
        R, length = log(64), log(200000)
        new = min(log(4096), 262144 // R)
        size = size_of(kv, h_q, R, new, length)
        for r, n, m in [(1, 1, length), (R, 1, length), (R, min(new, 16), length), (R, new, length)] + [
                (rng.randint(1, R), min(new, log(new + 1)), rng.randint(0, length)) for _ in range(20)]:
            for window in (0, log(200000)):
                assert enough(kv, h_q, size, r, n, m, window), (R, new, length, r, n, m, window)


def test_size_stays_in_proportion():
    """The query's answer is a bound, but not one that outgrows the parts there can be: unsplit
    sequences need none, and whatever the step at most 3200 workgroups of 32 rows."""
    kv = B.sfn_kv(1000, 16, 8, 128, 1, 0, FAKE, FAKE)
    assert size_of(kv, 32, 4, 1, 384) == B.SFN_WORKSPACE_HEADER_BYTES
    assert size_of(kv, 32, 1, 1, 1000) <= 2048 + 32 * 8 * 130 * 4 + 512
    assert size_of(kv, 1024, 4096, 64, 1 << 30) <= 2048 + 3200 * 32 * 130 * 4 + 512
