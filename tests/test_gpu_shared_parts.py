"""Where the parts of attention over a shared prefix lie, against the float64 oracle of each
request on its own: by request or by token, with tokens that no request has."""

import pytest

from tests.test_gpu_attend_shared import KINDS, after, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("own", [[(4000, 1), (20, 1), (700, 1)], [(4000, 5), (300, 0), (7, 1), (2100, 4)], [(900, 3), (40, 40), (5, 5)]],
                         ids=["one", "few", "many"])
@pytest.mark.parametrize("pad", [0, 200])
def test_parts_by_request_and_by_token(own, pad, dtype, kind):
    """As many tokens as the bounds allow, fewer, and (with `pad` behind the last) more; the own keys
    split and not."""
    check(dtype, kind, 8, 2, 128, 16, 500, after(500, own), seed=31, pad=pad)
    check(dtype, kind, 4, 4, 64, 64, 130, after(130, own), seed=32, pad=pad, apart=True)


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("max_new", [10 ** 3, 2 * 10 ** 5])
def test_bounds_far_above_the_tokens(max_new, dtype, kind):
    check(dtype, kind, 8, 2, 64, 16, 300, after(300, [(30, 3), (2000, 17), (9, 0), (65, 1)]), seed=33, max_new=max_new)
