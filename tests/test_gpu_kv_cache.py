"""The paged key/value cache on the GPU: the plan, the rotary append and the attention of
new tokens, against the float64 oracle."""

import random

import numpy as np
import pytest
import torch

from oracle import serving as S
from tests.helpers import say
from tests.serving_helpers import U32, UB, attend_bound, attend_oracle, f64, random_cache, rows_of, within

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from contextual_activation_sparsity_amd import binding as B

BF, F32 = torch.bfloat16, torch.float32


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def zeros(n):
    return torch.full((n,), -7, dtype=torch.int32, device="cuda")


# ---- plan ----------------------------------------------------------------------------


def run_plan(page, table, free, n_free, held, ctx, new, n_pages, max_tokens):
    kc = torch.zeros((n_pages, 1, page, 64), dtype=BF, device="cuda")
    o = dict(table=i32(table), free=i32(list(free) + [-1] * (n_pages - len(free))), n_out=zeros(1), cu=zeros(len(held) + 1),
             kv_len=zeros(len(held)), pos=zeros(max_tokens), slot=zeros(max_tokens), status=zeros(1))
    for _ in range(2):  # planning the same inputs again gives the same
        B.kv_cache_plan(B.KVCache(kc, kc), i32(held), i32(ctx), i32(new), o["table"], o["free"], i32([n_free]), o["n_out"], o["cu"],
                        o["kv_len"], o["pos"], o["slot"], o["status"])
    torch.cuda.synchronize()
    return {k: t.cpu().tolist() for k, t in o.items()}


def plan_case(rng, R, page, ctx_max, new_max, drop, free_extra):
    held = [rng.choice([0, 1, page - 1, page, page + 1, rng.randint(0, ctx_max)]) for _ in range(R)]
    kept = [rng.choice([h, max(0, h - rng.randint(0, drop)), 0]) for h in held]
    new = [rng.choice([0, 1, rng.randint(0, new_max)]) for _ in range(R)]
    up = lambda n: -(-n // page)  # noqa: E731
    cols = max([up(h) for h in held] + [up(c + n) for c, n in zip(kept, new)] + [1])
    takes = sum(max(0, up(c + n) - up(h)) for h, c, n in zip(held, kept, new))
    rels = sum(max(0, up(h) - up(c + n)) for h, c, n in zip(held, kept, new))
    n_free = max(0, takes - rels) + free_extra
    n_pages = sum(up(h) for h in held) + n_free
    order = list(range(max(n_pages, 1)))
    rng.shuffle(order)
    table, at = [], 0
    for h in held:
        table.append(order[at:at + up(h)] + [-9] * (cols - up(h)))
        at += up(h)
    return table, order[at:at + n_free], n_free, held, kept, new, max(n_pages, 1)


@pytest.mark.parametrize("R,page,ctx,new,drop,extra", [
    (1, 16, 40, 1, 0, 0), (1, 256, 1000, 300, 9, 2), (5, 16, 100, 7, 40, 0), (64, 32, 500, 1, 0, 3), (513, 16, 90, 5, 60, 0),
    (1030, 64, 200, 3, 200, 11), (4096, 16, 60, 2, 30, 5), (3, 128, 4000, 3000, 4000, 1)])
def test_plan_matches_the_oracle(R, page, ctx, new, drop, extra):
    rng = random.Random(R * 1000 + page)
    for rep in range(4):
        table, free, n_free, held, kept, nw, n_pages = plan_case(rng, R, page, ctx, new, drop, extra)
        spare = rng.choice([0, 5])
        max_tokens = max(1, sum(nw) + spare)
        say(f"[plan] R={R} page={page} rep={rep} tokens={sum(nw)}")
        want = S.cache_plan(page, table, free, n_free, held, kept, nw, n_pages, max_tokens)
        got = run_plan(page, table, free, n_free, held, kept, nw, n_pages, max_tokens)
        T = sum(nw)
        assert want["status"] == 0 and got["status"] == [0]
        assert got["cu"] == want["cu"] and got["kv_len"] == want["kv_len"]
        assert got["pos"][:T] == want["pos"] and got["slot"][:T] == want["slot"]
        assert got["pos"][T:] == [0] * (max_tokens - T) and got["slot"][T:] == [-1] * (max_tokens - T)
        assert got["n_out"] == [len(want["stack"])] and got["free"][:len(want["stack"])] == want["stack"]
        for r, used in enumerate(want["used"]):
            assert got["table"][r][:used] == want["table"][r][:used]


@pytest.mark.parametrize("held,ctx,new,free,status", [
    ([16], [16], [1], 0, 1), ([16, 16], [16, 16], [33, 1], 1, 3), ([16], [16], [49], 4, -1), ([16], [17], [1], 4, -1),
    ([-1], [0], [1], 4, -1), ([16], [-1], [1], 4, -1), ([16], [16], [-1], 4, -1), ([0, 0], [0, 0], [40, 40], 8, -1),
    ([2 ** 31 - 1], [2 ** 31 - 1], [2 ** 31 - 1], 4, -1)])
def test_plan_that_cannot_be_done_changes_nothing(held, ctx, new, free, status):
    table = [[1 + r, -9, -9, -9] for r in range(len(held))]
    stack = list(range(20, 20 + free))
    say(f"[plan refused] {held} {ctx} {new}")
    got = run_plan(16, table, stack, free, held, ctx, new, 32, 64)
    assert got["status"] == [status]
    assert got["table"] == table and got["free"][:free] == stack and got["n_out"] == [free]
    assert got["cu"] == [0] * (len(held) + 1) and got["kv_len"] == [0] * len(held)
    assert got["pos"] == [0] * 64 and got["slot"] == [-1] * 64


def test_plan_counts_of_pages_near_32_bits():
    R, page, cols, n_pages = 16, 16, 2 ** 27 - 1, 128
    table = torch.empty((R, cols), dtype=torch.int32, device="cuda")
    kc = torch.zeros((n_pages, 1, page, 64), dtype=BF, device="cuda")
    free, n_out, status = i32(list(range(n_pages))), zeros(1), zeros(1)
    say("[plan] given-back pages and free ones above 2^31 together")
    B.kv_cache_plan(B.KVCache(kc, kc), i32([cols * page] * R), i32([0] * R), i32([0] * R), table, free, i32([100]), n_out,
                    zeros(R + 1), zeros(R), zeros(4), zeros(4), status)
    assert status.item() == -1 and n_out.item() == 100
    assert free.tolist() == list(range(n_pages))


# ---- append --------------------------------------------------------------------------


def rope_table(n_pos, rot):
    ang = torch.arange(n_pos, dtype=torch.float64)[:, None] * (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot))[None]
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,h_q,h_kv,dh,page,rot", [
    (1, 32, 8, 128, 16, 128), (3, 7, 7, 64, 32, 64), (37, 28, 4, 128, 64, 64), (5, 0, 3, 64, 16, 32), (9, 4, 2, 128, 256, 48),
    (2, 5, 1, 64, 16, 0), (130, 1, 1, 128, 16, 16)])
def test_append_rotates_and_writes_its_slots_alone(dtype, T, h_q, h_kv, dh, page, rot):
    say(f"[append] {dtype} T={T} heads={h_q}/{h_kv} dh={dh} page={page} rot={rot}")
    g = torch.Generator().manual_seed(T * 100 + h_q)
    n_pages = T // page + 3
    qkv = torch.randn((T, h_q + 2 * h_kv + 1, dh), generator=g).to(dtype).cuda()  # one head more than is used: strided rows
    q, k, v = qkv[:, :h_q], qkv[:, h_q:h_q + h_kv], qkv[:, h_q + h_kv:h_q + 2 * h_kv]
    kc, vc = (torch.randn((n_pages, h_kv, page, dh), generator=g).to(dtype).cuda() for _ in range(2))
    k0, v0 = kc.clone(), vc.clone()
    slot = torch.randperm(n_pages * page, generator=g)[:T].to(torch.int32)
    if T > 2:
        slot[0], slot[2] = -1, n_pages * page  # these write nothing
    n_pos = 50
    pos = torch.randint(-3, 60, (T,), generator=g).to(torch.int32)
    rope = rope_table(n_pos, rot) if rot else None
    q_out = torch.full((T, h_q, dh), float("nan"), dtype=dtype, device="cuda")
    B.kv_cache_append(B.KVCache(kc, vc), k, v, slot.cuda(), q=q if h_q else None, q_out=q_out if h_q else None,
                      pos=pos.cuda() if rot else None, rope=rope.cuda() if rot else None)
    torch.cuda.synchronize()
    p = pos.numpy() if rot else np.zeros(T, int)
    tab = rope.numpy() if rot else np.zeros((1, 0))
    mag = lambda x: np.abs(x) + np.abs(np.roll(x, rot // 2, -1)) + np.abs(np.roll(x, -(rot // 2), -1))  # noqa: E731
    # two products and a sum in fp32, then the rounding; copies are exact
    if h_q:
        within(q_out, S.rotate(f64(q), p, tab, rot), UB[dtype] * np.abs(S.rotate(f64(q), p, tab, rot)) + 3 * U32 * mag(f64(q)), "q")
    want_k, want_v = f64(k0), f64(v0)
    kr = S.rotate(f64(k), p, tab, rot)
    bound = np.zeros_like(want_k)
    for t in range(T):
        s = int(slot[t])
        if 0 <= s < n_pages * page:
            want_k[s // page, :, s % page] = kr[t]
            want_v[s // page, :, s % page] = f64(v)[t]
            bound[s // page, :, s % page] = UB[dtype] * np.abs(kr[t]) + 3 * U32 * mag(f64(k)[t])
    within(kc, want_k, bound, "k")
    assert np.array_equal(f64(vc), want_v)


def test_append_in_place_and_empty():
    g = torch.Generator().manual_seed(1)
    q = torch.randn((4, 6, 64), generator=g).to(BF).cuda()
    k = torch.randn((4, 2, 64), generator=g).to(BF).cuda()
    kc = torch.zeros((2, 2, 16, 64), dtype=BF, device="cuda")
    cache = B.KVCache(kc, kc.clone())
    rope, pos, slot = rope_table(9, 64).cuda(), i32([1, 2, 3, 8]), i32([0, 1, 2, 3])
    out = torch.empty_like(q)
    B.kv_cache_append(cache, k, k, slot, q=q, q_out=out, pos=pos, rope=rope)
    B.kv_cache_append(cache, k, k, slot, q=q, q_out=q, pos=pos, rope=rope)
    B.kv_cache_append(cache, k[:0], k[:0], slot[:0])
    torch.cuda.synchronize()
    assert torch.equal(q, out)


# ---- attention -----------------------------------------------------------------------


def run_attend(q, k, v, table, cu, lens, window=0, max_new=None, max_len=None, scale=None, strided=False, stream=None):
    cache = B.KVCache(k.cuda(), v.cuda())
    R, (T, h_q, dh) = len(lens), q.shape
    max_new = max(1, max(b - a for a, b in zip(cu, cu[1:]))) if max_new is None else max_new
    max_len = max(lens) if max_len is None else max_len
    qd = q.cuda()
    if strided:
        wide = torch.full((T, h_q + 3, dh), float("nan"), dtype=q.dtype, device="cuda")
        wide[:, 1:h_q + 1] = qd
        qd = wide[:, 1:h_q + 1]
    out = torch.full((T, h_q, dh), float("nan"), dtype=q.dtype, device="cuda")
    ws = B.workspace(B.kv_cache_attend_workspace_size(cache, R, T, h_q, max_new, max_len))
    ws[2048:] = 255  # scratch is NaN: what is not written must not be read
    args = (cache, qd, table.cuda(), i32(cu), i32(lens), out, ws, max_new, max_len)
    B.kv_cache_attend(*args, scale=scale, window=window, stream=stream)
    torch.cuda.synchronize()
    first = out.clone()
    B.kv_cache_attend(*args, scale=scale, window=window, stream=stream)
    torch.cuda.synchronize()
    as_bits = torch.int16 if q.dtype == BF else torch.int32
    assert torch.equal(first.view(as_bits), out.view(as_bits)), "two runs differ"
    assert int(ws[:2048].to(torch.int32).sum()) == 0
    return out


def check_attend(dtype, h_q, h_kv, dh, page, reqs, window=0, seed=0, scale=None, std=1.0, **kw):
    """reqs: (kv_len, new tokens) of each request."""
    lens, news = [r[0] for r in reqs], [r[1] for r in reqs]
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    k, v, table = random_cache(lens, h_kv, dh, page, dtype, seed)
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn((cu[-1], h_q, dh), generator=g) * std).to(dtype)
    say(f"[attend] {dtype} heads={h_q}/{h_kv} dh={dh} page={page} window={window} reqs={reqs[:6]}")
    out = run_attend(q, k, v, table, cu, lens, window, scale=scale, **kw)
    sc = dh ** -0.5 if scale is None else scale
    for sl, want, bound in attend_oracle(q, k, v, table, cu, lens, window, sc):
        within(out[sl], want, bound, f"tokens {sl.start}..{sl.stop}")


HEADS = [(4, 4), (8, 2), (7, 1), (28, 4), (16, 1)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("h_q,h_kv", HEADS)
def test_attend_single_tokens_at_every_edge(dtype, dh, h_q, h_kv):
    """One token over 1, 2, ... keys around the edges of groups, tiles, pages and splits."""
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 700]
    for page in (16, 64, 256):
        check_attend(dtype, h_q, h_kv, dh, page, [(n, 1) for n in lens], seed=page)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("h_q,h_kv", HEADS)
def test_attend_chunks(dtype, dh, h_q, h_kv):
    """Chunks of 2 to 16 tokens, a prompt without a past among them, and requests without tokens."""
    reqs = [(16, 16), (5, 2), (0, 0), (130, 3), (33, 16), (300, 7), (64, 0), (65, 5), (17, 16), (1, 1)]
    check_attend(dtype, h_q, h_kv, dh, 16, reqs, seed=2)
    check_attend(dtype, h_q, h_kv, dh, 128, reqs, seed=3, strided=True)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("h_q,h_kv,dh,page,reqs", [
    (4, 2, 64, 16, [(150, 150), (61, 60), (400, 90)]), (6, 1, 128, 32, [(333, 333)]), (2, 2, 128, 256, [(513, 129), (128, 128), (127, 127)]),
    (8, 2, 128, 64, [(700, 37), (1, 1), (257, 256)]), (5, 1, 64, 64, [(260, 260)])])
def test_attend_prompts(dtype, h_q, h_kv, dh, page, reqs):
    check_attend(dtype, h_q, h_kv, dh, page, reqs, seed=4)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 33, 100, 1000])
def test_attend_windows(dtype, dh, window):
    check_attend(dtype, 8, 2, dh, 16, [(1, 1), (500, 1), (130, 16), (90, 90), (40, 5), (257, 100)], window=window, seed=window)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("h_q,h_kv", [(8, 2), (4, 4)])
def test_attend_rows_that_see_nothing(dtype, h_q, h_kv):
    """Sequences shorter than their new tokens, or empty: the first tokens see no key."""
    check_attend(dtype, h_q, h_kv, 128, 16, [(2, 5), (0, 3), (1, 20), (40, 40), (0, 1)], seed=6)
    check_attend(dtype, h_q, h_kv, 64, 32, [(0, 1)], seed=7, max_len=0)
    check_attend(dtype, h_q, h_kv, 64, 32, [(0, 1), (0, 200)], seed=7, max_len=512, window=3)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [1, 4, 16])
def test_attend_long_and_split(dtype, n):
    """Long sequences beside short ones: many splits, some of which a request does not reach."""
    check_attend(dtype, 4, 1, 128, 64, [(9000, n), (20, n), (4097, n)], seed=8)
    check_attend(dtype, 2, 2, 64, 16, [(6001, n)], seed=9, window=3500)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_sharp_and_flat_scores(dtype):
    """Scores of hundreds (one key takes all) and of nothing; a scale of its own."""
    check_attend(dtype, 4, 2, 128, 16, [(300, 1), (77, 40)], seed=10, std=60.0)
    check_attend(dtype, 4, 2, 64, 16, [(300, 1), (77, 40)], seed=11, std=0.0)
    check_attend(dtype, 4, 2, 64, 16, [(300, 1), (77, 40)], seed=12, scale=1.7)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("h_q,h_kv,n", [(2, 2, 8), (8, 2, 16), (6, 1, 100)])
def test_attend_tokens_do_not_see_later_infinities(dtype, h_q, h_kv, n):
    """NaN and infinite values of one token leave every earlier token's result as it was."""
    lens, cu, dh = [200], [0, n], 128
    k, v, table = random_cache(lens, h_kv, dh, 16, dtype, 13)
    q = torch.randn((n, h_q, dh), generator=torch.Generator().manual_seed(14)).to(dtype)
    say(f"[attend] infinities, {dtype} {h_q}/{h_kv} n={n}")
    clean = run_attend(q, k, v, table, cu, lens)
    bad = n // 2  # the token whose value is spoilt
    p = 200 - n + bad
    page, off = int(table[0, p // 16]), p % 16
    v[page, :, off, 3], v[page, :, off, 64], v[page, :, off, 127] = float("nan"), float("inf"), -float("inf")
    k[page, :, off, 5] = float("nan")
    out = run_attend(q, k, v, table, cu, lens)
    assert torch.equal(out[:bad], clean[:bad])
    assert torch.isnan(out[bad:]).all()
    k[page, :, off, 5] = 0.5
    out = run_attend(q, k, v, table, cu, lens)
    keep = [d for d in range(dh) if d not in (3, 64, 127)]
    assert torch.isfinite(out[bad:][..., keep]).all()
    assert torch.isnan(out[bad:][..., 3]).all() and (out[bad:][..., 64] == float("inf")).all() and (out[bad:][..., 127] == -float("inf")).all()


def test_attend_pages_out_of_range_stay_in_the_cache():
    k, v, table = random_cache([100], 2, 64, 16, BF, 15, poison=False)
    table[0, 1], table[0, 2] = -3, 2 ** 30
    q = torch.randn((1, 4, 64)).to(BF)
    out = run_attend(q, k, v, table, [0, 1], [100])
    fixed = table.clone()
    fixed[0, 1], fixed[0, 2] = 0, k.shape[0] - 1
    assert torch.equal(out, run_attend(q, k, v, fixed, [0, 1], [100]))


def test_attend_offsets_past_32_bits():
    """A cache of 5 GB a side whose pages lie at its end."""
    h_kv, page, dh, n_pages = 8, 64, 128, 40000
    k = torch.empty((n_pages, h_kv, page, dh), dtype=BF, device="cuda")
    v = torch.empty_like(k)
    assert k.numel() > 2 ** 31
    g = torch.Generator().manual_seed(16)
    pages = [39999, 0, 39990, 20000]
    small_k, small_v = (torch.randn((4, h_kv, page, dh), generator=g).to(BF) for _ in range(2))
    k[pages], v[pages] = small_k.cuda(), small_v.cuda()
    q = torch.randn((20, 16, dh), generator=g).to(BF)
    kn, vn = (torch.randn((20, h_kv, dh), generator=g).to(BF) for _ in range(2))
    slot = [p * page + o for p, o in zip([20000] * 20, range(44, 64))]
    B.kv_cache_append(B.KVCache(k, v), kn.cuda(), vn.cuda(), i32(slot))
    small_k[3, :, 44:], small_v[3, :, 44:] = kn.permute(1, 0, 2), vn.permute(1, 0, 2)
    cache = B.KVCache(k, v)
    for n in (1, 20):
        out = torch.empty((n, 16, dh), dtype=BF, device="cuda")
        ws = B.workspace(B.kv_cache_attend_workspace_size(cache, 1, n, 16, n, 256))
        B.kv_cache_attend(cache, q[-n:].cuda(), i32([pages]), i32([0, n]), i32([256]), out, ws, n, 256)
        torch.cuda.synchronize()
        table = torch.arange(4, dtype=torch.int32)[None]
        for _, want, bound in attend_oracle(q[-n:], small_k, small_v, table, [0, n], [256], 0, dh ** -0.5):
            within(out, want, bound, "long cache")


def test_attend_on_another_stream():
    lens, cu = [300, 40], [0, 1, 17]
    k, v, table = random_cache(lens, 2, 128, 16, BF, 17)
    q = torch.randn((17, 8, 128)).to(BF)
    here = run_attend(q, k, v, table, cu, lens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert torch.equal(here, run_attend(q, k, v, table, cu, lens, stream=s))


# ---- together ------------------------------------------------------------------------


@pytest.mark.parametrize("graphed", [False, True])
def test_steps_with_rollback_match_a_dense_cache(graphed):
    """Prompts, single tokens, a chunk of drafts, most of which the next step drops, and a
    request that ends: after every step the attention is that of the sequences kept on the
    host. In a graph, one capture serves every step of the same token count's bound."""
    g = torch.Generator().manual_seed(18)
    R, h_q, h_kv, dh, page, n_pages, cols, cap = 3, 8, 2, 64, 16, 24, 8, 64
    kc, vc = (torch.full((n_pages, h_kv, page, dh), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    cache = B.KVCache(kc, vc)
    rope = rope_table(200, dh).cuda()
    st = dict(held=i32([0] * R), ctx=i32([0] * R), new=i32([0] * R), table=i32([[-1] * cols] * R), free=i32(list(range(n_pages))),
              n=i32([n_pages]), n2=i32([0]), cu=i32([0] * (R + 1)), kv=i32([0] * R), pos=i32([0] * cap), slot=i32([0] * cap), status=i32([9]))
    qkv = torch.zeros((cap, h_q + 2 * h_kv, dh), dtype=BF, device="cuda")
    q_rot, out = (torch.zeros((cap, h_q, dh), dtype=BF, device="cuda") for _ in range(2))
    ws = B.workspace(B.kv_cache_attend_workspace_size(cache, R, cap, h_q, 48, 128))

    def step(stream=None):
        B.kv_cache_plan(cache, st["held"], st["ctx"], st["new"], st["table"], st["free"], st["n"], st["n2"], st["cu"], st["kv"],
                        st["pos"], st["slot"], st["status"], stream=stream)
        B.kv_cache_append(cache, qkv[:, h_q:h_q + h_kv], qkv[:, h_q + h_kv:], st["slot"], q=qkv[:, :h_q], q_out=q_rot, pos=st["pos"],
                          rope=rope, stream=stream)
        B.kv_cache_attend(cache, q_rot, st["table"], st["cu"], st["kv"], out, ws, 48, 128, stream=stream)

    graph = None
    if graphed:
        step()
        torch.cuda.synchronize()
        graph, cap_stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=cap_stream):
            step(cap_stream)
    seqs = [[] for _ in range(R)]  # the host's copy: (k, v) of each token kept, before rotation
    held = [0] * R
    plan = [([0, 0, 0], [40, 17, 0]), ([40, 17, 0], [1, 1, 6]), ([41, 18, 6], [16, 16, 16]), ([43, 34, 6], [1, 1, 1]), ([44, 0, 7], [16, 0, 16]),
            ([60, 0, 9], [1, 48, 1]), ([61, 48, 0], [1, 1, 0]), ([62, 49, 0], [1, 1, 30])]
    for n, (ctx, new) in enumerate(plan):
        say(f"[steps] graph={graphed} step {n}: keep {ctx}, new {new}")
        T = sum(new)
        qkv[:T] = torch.randn((T, h_q + 2 * h_kv, dh), generator=g).to(BF).cuda()
        st["held"].copy_(i32(held)), st["ctx"].copy_(i32(ctx)), st["new"].copy_(i32(new))
        out.fill_(float("nan"))
        graph.replay() if graphed else step()
        torch.cuda.synchronize()
        assert st["status"].item() == 0
        st["n"].copy_(st["n2"])
        host, t = qkv[:T].cpu(), 0
        for r in range(R):
            seqs[r] = seqs[r][:ctx[r]] + [(host[t + i, h_q:h_q + h_kv], host[t + i, h_q + h_kv:]) for i in range(new[r])]
            m = len(seqs[r])
            if new[r]:
                kk = rows_of(kc.cpu(), st["table"][r].cpu(), m)
                vv = torch.stack([x[1] for x in seqs[r]])
                pure = S.rotate(f64(torch.stack([x[0] for x in seqs[r]])), np.arange(m), rope.cpu().numpy(), dh)
                assert np.abs(f64(kk) - pure).max() <= 2.0 ** -8 * np.abs(pure).max()
                assert torch.equal(rows_of(vc.cpu(), st["table"][r].cpu(), m), vv)
                lo, hi = S.seen(m, new[r], 0)
                want, spread, reach = S.attend(f64(q_rot[t:t + new[r]]), f64(kk), f64(vv), lo, hi, dh ** -0.5)
                within(out[t:t + new[r]], want, attend_bound(want, spread, reach, m, dh, BF), f"step {n} request {r}")
            t += new[r]
        held = [c + x for c, x in zip(ctx, new)]
        used = sum(-(-h // page) for h in held)
        assert st["n"].item() == n_pages - used


# ---- every kernel variant ------------------------------------------------------------


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("window", [0, 130])
def test_attend_prompts_that_fill_the_chip(dh, window):
    """More than 256 row tiles of 128: one group of waves to a workgroup, no splits."""
    check_attend(BF, 16, 16, dh, 32, [(700, 650), (640, 640), (300, 129), (650, 650)], window=window, seed=20)


def test_attend_infinities_among_many_row_tiles():
    lens, cu = [650, 640], [0, 650, 1290]
    k, v, table = random_cache(lens, 32, 64, 64, BF, 21)
    q = torch.randn((1290, 32, 64), generator=torch.Generator().manual_seed(22)).to(BF)
    say("[attend] infinities among many row tiles")
    clean = run_attend(q, k, v, table, cu, lens)
    p = 300  # of the first request
    page, off = int(table[0, p // 64]), p % 64
    v[page, 5, off, 9] = float("inf")
    out = run_attend(q, k, v, table, cu, lens)
    same = torch.ones(out.shape, dtype=torch.bool, device="cuda")
    same[p:650, 5, 9] = False
    assert torch.equal(out[same], clean[same]) and (out[~same] == float("inf")).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [4, 16])
def test_attend_many_rows_with_splits(dtype, n):
    """Enough rows that a wave joins each, and several splits to join."""
    check_attend(dtype, 8, 2, 128, 64, [(2100, n), (1500, n), (60, n), (900, n)] * (4 if n == 4 else 1) + [(800, n)], seed=23)
    check_attend(dtype, 16, 4, 64, 16, [(1300, n), (1, 1), (777, n), (0, 0), (1024, n)], seed=24, window=900)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [1, 9])
def test_attend_unsplit_items_past_the_chip(dtype, n):
    """More unsplit requests than compute units: four waves to each, in one launch."""
    rng = random.Random(n)
    reqs = [(m + rng.choice([0, 1, rng.randint(0, 340)]), m) for m in (rng.choice([0, 1, n, n]) for _ in range(70))]
    check_attend(dtype, 8, 4, 64, 16, reqs, seed=27)
    check_attend(dtype, 10, 5, 128, 64, reqs, seed=28, window=100)


@pytest.mark.parametrize("lens", [[3000], [2900, 700]])
def test_attend_infinities_in_split_tiles(lens):
    """40 tokens of 8 / 1 heads over long sequences: tiles of 128 rows with split keys."""
    n, R = 40, len(lens)
    k, v, table = random_cache(lens, 1, 128, 32, BF, 29)
    q = torch.randn((n * R, 8, 128), generator=torch.Generator().manual_seed(30)).to(BF)
    say(f"[attend] infinities in split tiles {lens}")
    cu = [n * r for r in range(R + 1)]
    clean = run_attend(q, k, v, table, cu, lens)
    for sl, want, bound in attend_oracle(q, k, v, table, cu, lens, 0, 128 ** -0.5):
        within(clean[sl], want, bound, f"tokens {sl.start}..{sl.stop}")
    p = lens[0] - 17  # one of the first request's new tokens
    v[int(table[0, p // 32]), 0, p % 32, 77] = -float("inf")
    out = run_attend(q, k, v, table, cu, lens)
    same = torch.ones(out.shape, dtype=torch.bool, device="cuda")
    same[n - 17:n, :, 77] = False
    assert torch.equal(out[same], clean[same]) and (out[~same] == -float("inf")).all()


def test_attend_bounds_that_are_too_small():
    """Tokens past max_new are not computed (and not written), keys past max_len not read."""
    lens, cu = [90, 200], [0, 40, 60]
    for dtype, max_new in ((BF, 3), (F32, 9), (BF, 17)):
        k, v, table = random_cache(lens, 2, 128, 16, dtype, 25)
        q = torch.randn((60, 4, 128), generator=torch.Generator().manual_seed(26)).to(dtype)
        say(f"[attend] max_new {max_new} of 40 and 20, {dtype}")
        out = run_attend(q, k, v, table, cu, lens, max_new=max_new)
        for sl, want, bound in attend_oracle(q, k, v, table, cu, lens, 0, 128 ** -0.5):
            within(out[sl][:max_new], want[:max_new], bound[:max_new], "computed tokens")
            assert torch.isnan(out[sl][max_new:]).all()
    out = run_attend(q, k, v, table, cu, lens, max_len=100)
    cut = [90, 100]
    for sl, want, bound in attend_oracle(q, k, v, table, cu, cut, 0, 128 ** -0.5):
        within(out[sl], want, bound, "cut at 100 keys")


@pytest.mark.parametrize("seed", range(24))
def test_attend_drawn(seed):
    rng = random.Random(seed)
    h_q, h_kv = rng.choice([(4, 4), (8, 2), (7, 1), (28, 4), (16, 1), (12, 4), (3, 3)])
    reqs = []
    for _ in range(rng.randint(1, 9)):
        n = rng.choice([0, 1, 1, rng.randint(1, 16), rng.randint(1, 150)])
        reqs.append((n + rng.choice([0, rng.randint(0, 40), rng.randint(0, 1500)]), n))
    if not sum(n for _, n in reqs):
        reqs.append((17, 1))
    check_attend(rng.choice([BF, BF, F32]), h_q, h_kv, rng.choice([64, 128]), rng.choice([16, 32, 64, 128, 256]), reqs,
                 window=rng.choice([0, 0, rng.randint(1, 600)]), seed=seed, strided=rng.random() < 0.3)
