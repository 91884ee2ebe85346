"""Where the parts of attention over a shared prefix lie, against the float64 oracle of each
request on its own: by request or by token, with tokens that no request has, and with bounds that
are too small."""

import numpy as np
import pytest
import torch

from oracle import serving as S
from tests.helpers import say
from tests.serving_helpers import attend_bound, f64, rows_of, within
from tests.test_gpu_attend_shared import KINDS, Batch, after, check, tokens

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


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("h_q,h_kv", [(8, 2), (16, 1)])
def test_tokens_past_the_bound_take_no_place_of_others(h_q, h_kv, dtype, kind):
    """Requests with more tokens than the bound stand before others, which are computed as if the
    bound were right: in a step with more tokens than the bounds allow, and in one with fewer."""
    shared = 400
    for own, max_new in (([(60, 50), (9, 2), (33, 1), (70, 3)], 3), ([(5, 4), (9, 0), (33, 1), (70, 0)], 3), ([(200, 90), (90, 1)], 1),
                         ([(40, 20), (30, 0), (90, 0), (33, 33), (12, 7)], 8)):
        say(f"[shared] past the bound {max_new}, {dtype} {kind} {own}")
        b = Batch(dtype, kind, h_kv, 64, 16, shared, after(shared, own), 34)
        q = tokens(b, h_q, 64, 34)
        out = b.run(q, max_new=max_new, pad=11)
        for sl, want, bound in b.oracle(q):
            n = min(max_new, sl.stop - sl.start)
            within(out[sl][:n], want[:n], bound[:n], "computed tokens")
            assert out[sl][n:].isnan().all()


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_a_group_among_the_tokens_of_a_step(dtype, kind):
    """Single tokens behind one prompt, with other requests' tokens before and behind them, whose
    rows of the output stay as they are."""
    b = Batch(dtype, kind, 2, 128, 16, 3000, after(3000, [(40, 1), (1, 1), (260, 1)]), 35)
    q = torch.cat([tokens(b, 8, 128, 35 + i)[:n] for i, n in enumerate((3, 3, 3, 2))])
    alone = tokens(b, 8, 128, 36)
    q[5:8] = alone
    b.cu = [5 + c for c in b.cu]
    out = b.run(q, pad=300)
    b.cu = [c - 5 for c in b.cu]
    for sl, want, bound in b.oracle(alone):
        within(out[5:8][sl], want, bound, f"tokens {sl.start}..{sl.stop}")
    assert out[:5].isnan().all() and out[8:].isnan().all()


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("own", [[(60, 1), (1, 1), (900, 1)], [(45, 9), (200, 16)], [(90, 90), (150, 70)]], ids=["one", "chunks", "prompts"])
@pytest.mark.parametrize("shared,page", [(80, 16), (93, 32), (200, 256), (63, 64)])
def test_what_a_row_names_before_the_shared_tokens_end_changes_nothing(shared, page, own, dtype, kind):
    """Entries of the shared tokens' whole pages name the requests' own last pages, and the places of
    shared tokens in the page that the request goes on in hold NaN."""
    say(f"[shared] before the prefix's end {shared} page {page} {dtype} {kind} {own}")
    b = Batch(dtype, kind, 2, 128, page, shared, after(shared, own), 37)
    q = tokens(b, 8, 128, 37)
    want = b.run(q)
    for r in range(len(own)):
        at = int(b.table[r, shared // page])
        if kind == "e4m3":
            for codes, exps in b.cache.parts:
                codes.view(torch.uint8)[at, :, : shared % page], exps[at, :, : shared % page] = 255, 200
        else:
            b.k[at, :, : shared % page], b.v[at, :, : shared % page] = float("inf"), float("nan")
        b.table[r, : shared // page] = at
    assert torch.equal(b.run(q), want)


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("more", [0, 40])
@pytest.mark.parametrize("h_q,h_kv", [(8, 2), (4, 4)])
def test_tokens_before_the_first_offset_join_the_prefix_of_its_token(h_q, h_kv, more, dtype, kind):
    """Offsets that descend name tokens before cu[0], which the prefix's part, of [cu[0], cu[R]), is not
    made for. What they get is not for use, but it is made of parts that were written: their own
    keys' and, of the prefix, those of token cu[0]. Any other place would be before the prefix's parts."""
    shared, n, dh = 700, 2 + more, 64
    say(f"[shared] offsets that descend, {dtype} {kind} heads={h_q}/{h_kv} n={n}")
    b = Batch(dtype, kind, h_kv, dh, 16, shared, after(shared, [(20, 0), (30 + n, n), (40 + n, 2 * n)]), 3)
    b.cu = [2 * n, 0, n, 3 * n]
    q = tokens(b, h_q, dh, 3)
    out = b.run(q)
    first = np.broadcast_to(f64(q[2 * n]), (2 * n, h_q, dh))
    for r, t0, m in ((1, 0, n), (2, n, n)):
        past = b.lens[r] - b.news[r]
        if past < shared:  # of 40 more: it reads its own row alone
            row, cut = b.table[r], 0
        else:
            row, cut = torch.cat([b.prefix[: shared // 16], b.table[r, shared // 16:]]), shared
        k, v = (f64(rows_of(x, row, b.lens[r])) for x in (b.k, b.v))
        # queries of two parts, keys that meet one of them: the prefix's the first, the others the second
        none = np.zeros_like(k)
        k2 = np.concatenate([np.concatenate([k[:cut], none[:cut]], -1), np.concatenate([none[cut:], k[cut:]], -1)])
        q2 = np.concatenate([first[t0:t0 + m], f64(q[t0:t0 + m])], -1)
        want, spread, reach = S.attend(q2, k2, np.concatenate([v, v], -1), np.zeros(m), past + 1 + np.arange(m), dh ** -0.5)
        bound = attend_bound(want, spread, reach, b.lens[r], dh, dtype)
        within(out[t0:t0 + m], want[..., :dh], bound[..., :dh], f"tokens {t0}..{t0 + m}")
