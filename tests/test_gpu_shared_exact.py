"""Attention over a shared prefix is as exact as the same requests' without sharing."""

import math

import pytest
import torch

from tests.cache8_helpers import BF, F32, quantised
from tests.helpers import say

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from contextual_activation_sparsity_amd import binding as B


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("R,h_q,h_kv", [(3, 4, 1), (12, 4, 1), (12, 4, 4), (40, 8, 2)])
@pytest.mark.parametrize("dtype,kind", [(BF, "same"), (F32, "same"), (BF, "e4m3"), (F32, "e4m3")])
def test_weights_are_of_the_rows_largest_score(dtype, kind, R, h_q, h_kv, dh):
    """Scores (in log2) of 0 in every tile of 64 keys, and in every other one a key of 7.3125 whose
    values are 0.75 and one that has three quarters of its weight and values -1; all other weights
    are 0. Of the row's largest score the weights are 1, 3/4 and 2^-7.3125, and 1 and 3/4 are exact in
    bf16, so that each pair's values cancel exactly and so do all sums of them: the result is 0. With
    weights of any smaller score (a running maximum that lags) 2^7.3125 and 3/4 of it would be rounded
    apart, by up to 2^-8 of them."""
    say(f"[shared exact] {dtype} {kind} R={R} heads={h_q}/{h_kv} dh={dh}")
    page, tiles = 64, 600  # more tiles than there are splits, so that some split begins with a tile of score 0
    n_pages = tiles + R
    k, v = torch.zeros((n_pages, page, dh)), torch.zeros((n_pages, page, dh))
    k[:, :, 2] = 1.0  # a score that leaves no weight
    k[:tiles, 0, 2] = 0.0
    k[1:tiles:2, 5, :3] = torch.tensor([1.0, 0.0, 0.0])
    k[1:tiles:2, 21, :4] = torch.tensor([0.0, 1.0, 0.0, 1.0])
    v[1:tiles:2, 5], v[1:tiles:2, 21] = 0.75, -1.0
    v[tiles:] = 1.0  # the requests' own tokens
    k, v = (x[:, None].expand(n_pages, h_kv, page, dh).contiguous() for x in (k, v))
    q = torch.zeros((R, h_q, dh))
    lower = 7.3125 - math.log2(4 / 3)  # in two bf16 values
    hi = torch.tensor(lower).to(BF).item()
    q[:, :, 0], q[:, :, 1], q[:, :, 2], q[:, :, 3] = 7.3125, hi, -1000.0, torch.tensor(lower - hi).to(BF).item()
    q = q.to(dtype).cuda()
    if kind == "e4m3":
        (kc, kb), (vc, vb) = quantised(k), quantised(v)
        cache = B.KVCache8(kc.cuda(), vc.cuda(), kb.cuda(), vb.cuda(), dtype)
        plain, plain_size = B.kv8_cache_attend, B.kv8_cache_attend_workspace_size
        call, size = B.kv8_cache_attend_shared, B.kv8_cache_attend_shared_workspace_size
    else:
        cache = B.KVCache(k.to(dtype).cuda(), v.to(dtype).cuda())
        plain, plain_size = B.kv_cache_attend, B.kv_cache_attend_workspace_size
        call, size = B.kv_cache_attend_shared, B.kv_cache_attend_shared_workspace_size
    shared, n = tiles * page, tiles * page + 1
    prefix = i32(list(range(tiles)))
    table = torch.cat([prefix.expand(R, tiles), i32([[tiles + r] for r in range(R)])], 1).contiguous()
    cu, lens = i32(list(range(R + 1))), i32([n] * R)
    ws = B.workspace(max(size(cache, R, R, h_q, 1, shared, 1), plain_size(cache, R, R, h_q, 1, n)))
    for what in ("each on its own", "shared"):
        out = torch.full((R, h_q, dh), float("nan"), dtype=dtype, device="cuda")
        if what == "shared":
            call(cache, q, prefix, i32([shared]), table, cu, lens, out, ws, 1, shared, 1, scale=math.log(2))
        else:
            plain(cache, q, table, cu, lens, out, ws, 1, n, scale=math.log(2))
        torch.cuda.synchronize()
        # fp32 does not round the weights: 3/4 is off by what its score and the exponential are
        most = 0.0 if dtype == BF else 2.0 ** -14
        assert out.abs().max().item() <= most, (what, out.abs().max().item())
