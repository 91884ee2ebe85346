"""Rows of the 8-bit cache read back and appended again, codes and bytes against the oracle."""

import numpy as np
import pytest
import torch

from oracle import serving as S
from tests.cache8_helpers import BF, E4M3, F32
from tests.helpers import say
from tests.serving_helpers import f64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from contextual_activation_sparsity_amd import binding as B


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dh", [64, 128])
def test_the_same_values_with_the_oracles_codes(dtype, dh):
    say(f"[cache8 again] {dtype} dh={dh}")
    g = torch.Generator().manual_seed(dh)
    T, h_kv, page = 48, 3, 16
    rows = [torch.randn((T, h_kv, dh), generator=g) for _ in range(2)]
    for x in rows:  # largest magnitudes about the one that is rounded down to 1.75 times a power of two
        top = torch.linspace(1.7, 1.9, T * h_kv).view(T, h_kv) * 2.0 ** torch.randint(-20, 20, (T, h_kv), generator=g)
        x *= (top * 0.99 / x.abs().amax(-1))[..., None]
        x[..., 5] = top
    k, v = (x.to(dtype).cuda() for x in rows)
    slot = torch.randperm(T, generator=g).to(torch.int32).cuda()

    def cache():
        codes = [torch.full((T // page, h_kv, page, dh), 77, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
        return B.KVCache8(*codes, *(torch.full((T // page, h_kv, page), 99, dtype=torch.uint8, device="cuda") for _ in range(2)), dtype)

    first, second = cache(), cache()
    got = [[torch.empty_like(k) for _ in range(2)] for _ in range(2)]
    B.kv8_cache_append(first, k, v, slot)
    B.kv8_cache_read(first, slot, *got[0])
    B.kv8_cache_append(second, *got[0], slot)
    B.kv8_cache_read(second, slot, *got[1])
    torch.cuda.synchronize()
    at = slot.cpu().long()
    lower = 0
    for x, a, b, codes, exps, exps1 in ((k, got[0][0], got[1][0], second.k, second.k_exp, first.k_exp),
                                        (v, got[0][1], got[1][1], second.v, second.v_exp, first.v_exp)):
        assert torch.equal(a, b)
        c1, b1 = S.quantise(f64(x))
        c2, b2 = S.quantise(S.stand_for(c1, b1))
        rows_at = lambda t: t.cpu().view(torch.uint8)[at // page, :, at % page].numpy()  # noqa: E731
        assert np.array_equal(rows_at(exps1), b1) and np.array_equal(rows_at(exps), b2) and np.array_equal(rows_at(codes), c2)
        lower += int((b1 != b2).sum())
    assert lower > 0
