"""The paged cache's calls at their bounds on the GPU: workspaces of a program's largest step,
lengths past the bounds, counts that do not fit, splits up to the most there are."""

import numpy as np
import pytest
import torch

from oracle import serving as S
from tests.helpers import say
from tests.serving_helpers import attend_oracle, f64, random_cache, within
from tests.test_gpu_draft_and_verify import full_logits, load
from tests.test_gpu_kv_cache import check_attend, i32, run_attend, run_plan

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from contextual_activation_sparsity_amd import binding as B

BF, F32 = torch.bfloat16, torch.float32


def test_one_workspace_for_long_sequences_serves_every_step():
    """The example's workspace is sized for its longest prompts; its single tokens and chunks,
    whose keys are split where a prompt's are not, have to fit into it. The bound is the one of
    test_prompt_chunk_and_single_token_logits_match_float64."""
    m = load()
    model = m.Decoder(max_len=4080)
    g = np.random.default_rng(1)
    seqs = [g.integers(0, 500, n).tolist() for n in (50, 31, 44)]
    want = [full_logits(model, s) for s in seqs]
    say("[example] long bounds")
    model.step([s[:20] for s in seqs], [0, 0, 0], dense=True)
    chunk = f64(model.step([s[20:30] for s in seqs], [20, 20, 20], dense=True))
    one = f64(model.step([s[30:31] for s in seqs], [30, 30, 30], dense=True))
    assert model.status.item() == 0
    for r in range(3):
        top = np.abs(want[r]).max()
        assert np.abs(chunk[10 * r:10 * r + 10] - want[r][20:30]).max() < 1e-3 * top
        assert np.abs(one[r] - want[r][30]).max() < 1e-3 * top


def test_norm_rows_of_another_length_are_refused():
    """[4, 32] is not two rows of 64, nor [2, 128] four of them."""
    bf = dict(dtype=BF, device="cuda")
    norm = B.ResidualNorm(torch.ones(64, **bf))
    h, y, x = torch.ones((4, 64), **bf), torch.ones((4, 64), **bf), torch.zeros((4, 64), **bf)
    wrong = [torch.ones((8, 32), **bf), torch.ones((2, 128), **bf), torch.ones(256, **bf), torch.ones((64, 4), **bf)]
    for w in wrong:
        for name, args, kw in (("h", (w, None, None, x), {}), ("y", (h, w, None, x), {}), ("gate", (h, y, None, x), dict(gate=w))):
            with pytest.raises(ValueError, match=rf"{name} must be \[T, 64\]"):
                B.residual_norm(norm, *args, **kw)
    # rows over more dimensions, one row alone, and a longer buffer's first rows stay as they were
    B.residual_norm(norm, h, y, None, x)
    again = torch.zeros_like(x)
    B.residual_norm(norm, h.view(2, 2, 64), torch.cat([y, y]), None, again, gate=torch.ones(64, **bf))
    one = torch.zeros(64, **bf)
    B.residual_norm(norm, h[0], y[0], None, one)
    torch.cuda.synchronize()
    assert torch.equal(x, again) and torch.equal(one, x[0])


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("scale", [None, 2.0])
def test_attend_two_groups_join(dh, scale):
    """Tiles of 128 rows whose keys two groups of waves share, split and whole, with stages for
    both, for one alone, and maxima far apart (one group's sums all but vanish): each wave's
    rows go through the LDS that it has just read the other group's sums from."""
    for reqs in ([(700, 16), (129, 16), (64, 16), (65, 16)], [(16, 16)], [(130, 100), (1000, 100)], [(5000, 24), (40, 40)]):
        check_attend(BF, 16, 2, dh, 64, reqs, seed=31, scale=scale)
        check_attend(BF, 9, 1, dh, 16, reqs, seed=32, scale=scale, window=150)


@pytest.mark.parametrize("n_free", [-1, -2 ** 31, 9, 2 ** 31 - 1])
@pytest.mark.parametrize("held,ctx,new", [([16], [16], [1]), ([16], [3], [1]), ([32], [0], [0])])
def test_plan_with_a_count_of_free_pages_that_cannot_be(n_free, held, ctx, new):
    """Of 8 pages: refused as a whole, the count handed on as it came."""
    say(f"[plan] n_free {n_free} {held} {ctx} {new}")
    table, stack = [[1, 2, -9, -9]], [3, 4, 5, 6, 7, 0]
    assert S.cache_plan(16, table, stack, n_free, held, ctx, new, 8, 4) == {"status": -1}
    got = run_plan(16, table, stack, n_free, held, ctx, new, 8, 4)
    assert got["status"] == [-1] and got["n_out"] == [n_free]
    assert got["table"] == table and got["free"] == stack + [-1, -1]
    assert got["cu"] == [0, 0] and got["kv_len"] == [0] and got["pos"] == [0] * 4 and got["slot"] == [-1] * 4


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [0, 60])
@pytest.mark.parametrize("lens,cu,h_q,max_len,cols", [
    ([200, 90], [0, 20, 23], 4, 100, None), ([200, 90], [0, 150, 153], 4, 100, None), ([1900, 700], [0, 30, 31], 8, 1000, None),
    ([900, 40], [0, 1, 2], 4, 900, 33), ([900, 40], [0, 100, 101], 16, 2 ** 30, 33)])
def test_attend_of_requests_past_a_bound_is_of_the_shorter_request(dtype, window, lens, cu, h_q, max_len, cols):
    """kv_len past max_len, or past a table row of `cols` pages, counts as that bound: positions,
    causal limits and windows are the shorter request's, in every kernel."""
    k, v, table = random_cache(lens, 2, 64, 16, dtype, 33)
    if cols:
        table = table[:, :cols].contiguous()
    q = torch.randn((cu[-1], h_q, 64), generator=torch.Generator().manual_seed(34)).to(dtype)
    say(f"[attend] past the bounds, {dtype} window={window} {lens} max_len={max_len} cols={cols}")
    out = run_attend(q, k, v, table, cu, lens, window, max_len=max_len)
    cut = [min(n, max_len, 16 * table.shape[1]) for n in lens]
    assert cut[0] < lens[0]
    for sl, want, bound in attend_oracle(q, k, v, table, cu, cut, window, 64 ** -0.5):
        within(out[sl], want, bound, f"tokens {sl.start}..{sl.stop}")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_tokens_past_max_new_leave_the_others(dtype):
    """max_new too small: the tokens that are computed have their own positions."""
    lens, cu = [300, 120], [0, 40, 45]
    k, v, table = random_cache(lens, 2, 64, 16, dtype, 35)
    q = torch.randn((45, 4, 64), generator=torch.Generator().manual_seed(36)).to(dtype)
    for max_new, window in ((1, 0), (7, 50), (39, 0)):
        say(f"[attend] max_new {max_new} window {window} {dtype}")
        out = run_attend(q, k, v, table, cu, lens, window, max_new=max_new)
        for sl, want, bound in attend_oracle(q, k, v, table, cu, lens, window, 64 ** -0.5):
            within(out[sl][:max_new], want[:max_new], bound[:max_new], "computed tokens")
            assert torch.isnan(out[sl][max_new:]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_of_some_requests_at_a_time(dtype):
    """A step of prompts, chunks and single tokens in a call for each kind: parts of the page
    table, of cu (offsets into all tokens) and of the lengths, one output."""
    lens, news = [900, 33, 1500, 1, 70, 260, 420], [1, 1, 1, 1, 16, 9, 200]
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    k, v, table = random_cache(lens, 2, 128, 32, dtype, 37)
    q = torch.randn((cu[-1], 8, 128), generator=torch.Generator().manual_seed(38)).to(dtype)
    cache, qd, td, cd, ld = B.KVCache(k.cuda(), v.cuda()), q.cuda(), table.cuda(), i32(cu), i32(lens)
    out = torch.full(q.shape, float("nan"), dtype=dtype, device="cuda")
    ws = B.workspace(B.kv_cache_attend_workspace_size(cache, len(lens), cu[-1], 8, 200, 1500))
    for r0, r1, n in ((0, 4, 1), (4, 6, 16), (6, 7, 200)):
        say(f"[attend] requests {r0} to {r1} of a mixed step, {dtype}")
        B.kv_cache_attend(cache, qd, td[r0:r1], cd[r0:r1 + 1], ld[r0:r1], out, ws, n, 1500)
    torch.cuda.synchronize()
    for sl, want, bound in attend_oracle(q, k, v, table, cu, lens, 0, 128 ** -0.5):
        within(out[sl], want, bound, f"tokens {sl.start}..{sl.stop}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dh,n_keys", [(64, 9500), (64, 20001), (64, 32768), (128, 32768)])
def test_attend_most_splits(dtype, dh, n_keys):
    """One token of one head over a long sequence: up to the 256 splits that there are at most,
    for which the join reads its parts in several rounds."""
    check_attend(dtype, 1, 1, dh, 64, [(n_keys, 1)], seed=39)
    check_attend(dtype, 2, 1, dh, 64, [(n_keys, 3)], seed=40)


def test_example_refuses_sequences_past_its_tables():
    """A plan that cannot be done leaves the step without tokens, and its logits without meaning:
    the example stops before it. 36 tokens and 16 drafts past them fill a table of 52."""
    m = load()
    model = m.Decoder(max_len=52, requests=2)
    seqs, _, _ = model.generate([[1, 2, 3], [4] * 30], 6)
    assert [len(s) for s in seqs] == [9, 36] and model.status.item() == 0
    model = m.Decoder(max_len=44, requests=2)
    with pytest.raises(ValueError, match="max_len = 44"):
        model.generate([[1, 2, 3], [4] * 30], 6)
