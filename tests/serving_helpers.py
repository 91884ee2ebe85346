"""Inputs and error bounds shared by the tests of the paged cache and the residual norm."""

import numpy as np
import torch

from oracle import serving as S

U32 = 2.0 ** -24
UB = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # one rounding to the type
LAMBDA = 8.0  # a sum of n rounded terms errs by at most LAMBDA u sqrt(n) |terms|_2, but for odds below exp(-32)


def f64(t):
    return t.detach().double().cpu().numpy()


def attend_bound(out, spread, reach, n_keys, dh, dtype):
    """Elementwise bound of the attention's error from the rounding it does.

    A score errs by ds = LAMBDA u sqrt(dh) |q k|_2 for its products and sum, plus a few
    roundings of the score itself, of the exponent's argument and of the exponential; a weight
    by the factor 1 + 2 ds at most, as its row's sum errs too (ds << 1); sums over the keys, in
    fp32, by LAMBDA u sqrt(keys). bf16 rounds each weight once more (2^-8 of it), and the
    result. Each acts on sum_j w_j |v_j| (spread), the last on the result alone."""
    ds = U32 * (LAMBDA * np.sqrt(dh) * reach[..., :1] + 8.0 * reach[..., 1:] + 16.0)
    rel = 2.0 * ds + U32 * (LAMBDA * np.sqrt(max(n_keys, 1)) + 16.0)
    if dtype == torch.bfloat16:
        rel = rel + UB[dtype]
    return rel * spread + UB[dtype] * np.abs(out) + 1e-30


def within(got, want, bound, what):
    got, bad = f64(got), None
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.isfinite(got).all(), f"{what}: {np.count_nonzero(~np.isfinite(got))} values are not finite"
    over = np.abs(got - want) - bound
    if (over > 0).any():
        bad = np.unravel_index(np.argmax(over), over.shape)
    assert bad is None, f"{what}: at {bad} {got[bad]} for {want[bad]}, bound {np.broadcast_to(bound, want.shape)[bad]}"


def random_cache(lens, h_kv, dh, page, dtype, seed, spare=3, poison=True, extra_cols=2):
    """A cache whose requests hold lens[r] tokens on shuffled pages, and a table with rubbish in
    the entries no request uses. Places that hold no token are NaN when poisoned."""
    g = torch.Generator().manual_seed(seed)
    pages = [-(-n // page) for n in lens]
    n_pages = sum(pages) + spare
    order = torch.randperm(n_pages, generator=g).tolist()
    cols = max(pages + [1]) + extra_cols
    table = torch.full((len(lens), cols), 2 ** 31 - 1, dtype=torch.int32)
    table[:, 1::2] = -5
    fill = float("nan") if poison else 0.0
    k = torch.full((n_pages, h_kv, page, dh), fill, dtype=torch.float32)
    v = torch.full((n_pages, h_kv, page, dh), fill, dtype=torch.float32)
    at = 0
    for r, n in enumerate(lens):
        own = order[at:at + pages[r]]
        at += pages[r]
        table[r, :len(own)] = torch.tensor(own, dtype=torch.int32)
        for i, p in enumerate(own):
            m = min(page, n - i * page)
            k[p, :, :m] = torch.randn((h_kv, m, dh), generator=g)
            v[p, :, :m] = torch.randn((h_kv, m, dh), generator=g)
    return k.to(dtype), v.to(dtype), table


def rows_of(cache, table_row, n):
    """The n tokens of a request, [n, h_kv, dh], from a cache on the host."""
    page = cache.shape[2]
    own = table_row[: -(-n // page)].long()
    return cache[own].permute(0, 2, 1, 3).reshape(-1, cache.shape[1], cache.shape[3])[:n]


def attend_oracle(q, k, v, table, cu, lens, window, scale):
    """Per request: (slice, out, bound) of every token that the call computes."""
    dh = q.shape[2]
    for r, n_len in enumerate(lens):
        t0, t1 = cu[r], cu[r + 1]
        lo, hi = S.seen(n_len, t1 - t0, window)
        kk, vv = rows_of(k, table[r], n_len), rows_of(v, table[r], n_len)
        out, spread, reach = S.attend(f64(q[t0:t1]), f64(kk), f64(vv), lo, hi, scale)
        yield slice(t0, t1), out, attend_bound(out, spread, reach, n_len, dh, q.dtype)
