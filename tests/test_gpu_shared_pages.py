"""Pages that several rows name, and the plan, on the GPU: requests that end and start over as the
header says keep the prefix's pages until it is over."""

import pytest
import torch

from tests import shared_pages as P
from tests.helpers import say

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from contextual_activation_sparsity_amd import binding as B


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("e8", [False, True])
def test_requests_that_end_at_the_shared_pages_lose_none(e8):
    shape = (P.N_PAGES, 2, P.PAGE, 64)
    if e8:
        codes, b = torch.zeros(shape, dtype=torch.float8_e4m3fn, device="cuda"), torch.zeros(shape[:3], dtype=torch.uint8, device="cuda")
        cache = B.KVCache8(codes, codes.clone(), b, b.clone())
    else:
        cache = B.KVCache(*(torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    free = [p for p in range(P.N_PAGES) if p not in P.PREFIX]
    table, stack, n = i32([P.PREFIX + [-1] * (P.COLS - len(P.PREFIX))] * P.ROWS), i32(free + [-1] * len(P.PREFIX)), i32([len(free)])
    n2, cu, kv_len, pos, slot, status = i32([0]), i32([0] * (P.ROWS + 1)), i32([0] * P.ROWS), i32([0] * 100), i32([0] * 100), i32([9])
    for i, step in enumerate(P.STEPS):
        say(f"[shared pages] step {i} {step}")
        held, ctx, new = P.tokens(step)
        B.kv_cache_plan(cache, i32(held), i32(ctx), i32(new), table, stack, n, n2, cu, kv_len, pos, slot, status)
        torch.cuda.synchronize()
        assert status.item() == 0
        n.copy_(n2)
        used = [-(-(c + x) // P.PAGE) for c, x in zip(ctx, new)]
        P.check([row[:u] for row, u in zip(table.tolist(), used)], stack.tolist()[:n.item()], shared=i < 6)
