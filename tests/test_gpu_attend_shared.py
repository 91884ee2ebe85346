"""Attention over a shared prefix on the GPU, for caches in the tokens' type and in 8 bits,
against the float64 oracle of each request on its own."""

import random

import numpy as np
import pytest
import torch

from oracle import serving as S
from tests.cache8_helpers import BF, E4M3, F32, Cache8, values
from tests.helpers import say
from tests.serving_helpers import attend_bound, attend_oracle, f64, random_cache, rows_of, within

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from contextual_activation_sparsity_amd import binding as B

KINDS = [(BF, "same"), (F32, "same"), (BF, "e4m3"), (F32, "e4m3")]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cu_of(news):
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    return cu


class Batch:
    """Requests whose first `shared` tokens are the same: the host's cache, its tables, and the
    pages of the prefix. The prefix's whole pages stand in every row, or, where `apart`, in none
    (entries that no one may read are rubbish); a page that it fills in part is in each request's
    row with the same tokens."""

    def __init__(self, dtype, kind, h_kv, dh, page, shared, reqs, seed, apart=False, extra_cols=2):
        self.dtype, self.kind, self.shared, self.page = dtype, kind, shared, page
        self.lens, self.news = [r[0] for r in reqs], [r[1] for r in reqs]
        self.cu = cu_of(self.news)
        k, v, table = random_cache([shared] + self.lens, h_kv, dh, page, F32, seed, extra_cols=extra_cols)
        whole = shared // page
        self.prefix = table[0, : max(1, -(-shared // page))].clone()
        if shared == 0:
            self.prefix[:] = -9
        self.table = table[1:].clone()
        for r, n in enumerate(self.lens):
            past = n - self.news[r]
            for p in range(min(shared, n)):
                a, b = int(self.prefix[p // page]), int(self.table[r, p // page])
                k[b, :, p % page], v[b, :, p % page] = k[a, :, p % page], v[a, :, p % page]
            if whole and past >= shared:  # its own copy of the whole pages is not to be read
                for e in range(whole):
                    own = int(self.table[r, e])
                    k[own], v[own] = float("nan"), float("nan")
                    self.table[r, e] = 2 ** 31 - 1 if apart else self.prefix[e]
        if kind == "e4m3":
            self.cache = Cache8(k, v, seed)
            self.k, self.v = self.cache.k, self.cache.v
        else:
            self.k, self.v = k.to(dtype), v.to(dtype)
        self.own = max([n - shared if n - m >= shared else n for n, m in reqs] + [0])

    def handle(self):
        return self.cache.on_gpu(B, self.dtype) if self.kind == "e4m3" else B.KVCache(self.k.cuda(), self.v.cuda())

    def calls(self):
        return ((B.kv8_cache_attend_shared, B.kv8_cache_attend_shared_workspace_size) if self.kind == "e4m3" else
                (B.kv_cache_attend_shared, B.kv_cache_attend_shared_workspace_size))

    def oracle(self, q, scale=None, lens=None):
        """Each request on its own, its whole sequence in its own row: the prefix's pages in front of the rest."""
        table, whole = self.table.clone(), self.shared // self.page
        for r, n in enumerate(self.lens):
            if n - self.news[r] >= self.shared:
                table[r, :whole] = self.prefix[:whole]
        return attend_oracle(q, self.k, self.v, table, self.cu, lens or self.lens, 0, q.shape[2] ** -0.5 if scale is None else scale)

    def run(self, q, max_new=None, max_shared=None, max_own=None, scale=None, strided=False, stream=None, pad=0):
        call, size = self.calls()
        R, (T, h_q, dh) = len(self.lens), q.shape
        max_new = max(1, max(self.news)) if max_new is None else max_new
        max_shared, max_own = self.shared if max_shared is None else max_shared, self.own if max_own is None else max_own
        qd = torch.cat([q, torch.full((pad, h_q, dh), float("nan"), dtype=q.dtype)]).cuda()
        T += pad
        if strided:
            wide = torch.full((T, h_q + 3, dh), float("nan"), dtype=q.dtype, device="cuda")
            wide[:, 1:h_q + 1] = qd
            qd = wide[:, 1:h_q + 1]
        out = torch.full((T, h_q, dh), float("nan"), dtype=q.dtype, device="cuda")
        cache = self.handle()
        ws = B.workspace(size(cache, R, T, h_q, max_new, max_shared, max_own))
        ws[2048:] = 255  # scratch is NaN: what is not written must not be read
        args = (cache, qd, self.prefix.cuda(), i32([self.shared]), self.table.cuda(), i32(self.cu), i32(self.lens), out, ws, max_new, max_shared,
                max_own)
        call(*args, scale=scale, stream=stream)
        torch.cuda.synchronize()
        first = out.clone()
        call(*args, scale=scale, stream=stream)
        torch.cuda.synchronize()
        as_bits = torch.int16 if q.dtype == BF else torch.int32
        assert torch.equal(first.view(as_bits), out.view(as_bits)), "two runs differ"
        assert int(ws[:2048].to(torch.int32).sum()) == 0
        assert torch.isnan(out[T - pad:]).all()
        return out[:T - pad]


def tokens(batch, h_q, dh, seed, std=1.0):
    return (torch.randn((batch.cu[-1], h_q, dh), generator=torch.Generator().manual_seed(seed + 1)) * std).to(batch.dtype)


def check(dtype, kind, h_q, h_kv, dh, page, shared, reqs, seed=0, scale=None, std=1.0, apart=False, **kw):
    """reqs: (kv_len, new tokens) of each request, the shared tokens counted."""
    say(f"[shared] {dtype} {kind} heads={h_q}/{h_kv} dh={dh} page={page} shared={shared} reqs={reqs[:6]}")
    b = Batch(dtype, kind, h_kv, dh, page, shared, reqs, seed, apart)
    q = tokens(b, h_q, dh, seed, std)
    out = b.run(q, scale=scale, **kw)
    for sl, want, bound in b.oracle(q, scale):
        within(out[sl], want, bound, f"tokens {sl.start}..{sl.stop}")


def after(shared, own):
    """Requests with `own` (tokens after the prefix, new tokens of them)."""
    return [(shared + n, m) for n, m in own]


EDGES = [(1, 1), (2, 1), (15, 1), (16, 1), (17, 1), (33, 1), (64, 1), (65, 1), (130, 1), (300, 1), (411, 1)]


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("h_q,h_kv", [(4, 4), (8, 2), (7, 1)])
@pytest.mark.parametrize("shared", [0, 1, 16, 63, 64, 129, 500])
def test_single_tokens_at_every_edge(dtype, kind, dh, h_q, h_kv, shared):
    check(dtype, kind, h_q, h_kv, dh, 16, shared, after(shared, EDGES), seed=shared)
    check(dtype, kind, h_q, h_kv, dh, 64, shared, after(shared, EDGES[:2]), seed=shared + 1, apart=True)


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("h_q,h_kv,dh,page", [(4, 4, 64, 16), (8, 2, 128, 128), (28, 4, 128, 32), (16, 1, 64, 256)])
def test_chunks_and_prompts(dtype, kind, h_q, h_kv, dh, page):
    """Chunks, prompts and requests without tokens, strided queries, rows behind the last token."""
    own = [(16, 16), (5, 2), (0, 0), (130, 3), (33, 16), (64, 0), (65, 5), (1, 1)]
    check(dtype, kind, h_q, h_kv, dh, page, 257, after(257, own), seed=2, strided=True, pad=5)
    check(dtype, kind, h_q, h_kv, dh, page, 100, after(100, [(90, 90), (150, 149), (40, 7)]), seed=3, apart=True)


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_requests_that_do_not_come_after_the_prefix(dtype, kind):
    """Shorter than the shared tokens, within them, empty, or longer but not after: they read
    their own rows, and rows that see no key give zeros."""
    shared = 100
    reqs = [(130, 30), (130, 31), (100, 1), (99, 1), (3, 3), (0, 0), (2, 5), (0, 2), (101, 1), (300, 20), (100, 0), (40, 0), (116, 16)]
    check(dtype, kind, 8, 2, 128, 16, shared, reqs, seed=4)
    check(dtype, kind, 4, 4, 64, 64, shared, reqs, seed=5)
    check(dtype, kind, 4, 2, 64, 32, shared, [(99, 1), (20, 4), (0, 0)], seed=6)  # nobody comes after it


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("n", [1, 3, 16])
def test_long_prefixes_and_splits(dtype, kind, n):
    check(dtype, kind, 4, 1, 128, 64, 6000, after(6000, [(3000, n), (20, n), (1097, n)]), seed=8)
    check(dtype, kind, 2, 2, 64, 16, 5001, after(5001, [(n, n), (700, n)]), seed=9)
    check(dtype, kind, 8, 1, 64, 16, 40, after(40, [(n, n), (4000, n)]), seed=9)


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_many_requests(dtype, kind):
    rng = random.Random(3)
    check(dtype, kind, 8, 4, 64, 16, 300, after(300, [(rng.randint(1, 60), 1) for _ in range(150)]), seed=10)
    own = [(n + rng.randint(0, 100), n) for n in (rng.randint(0, 12) for _ in range(40))]
    check(dtype, kind, 8, 2, 128, 32, 700, after(700, own), seed=11)


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_sharp_and_flat_scores(dtype, kind):
    for std, scale in ((60.0, None), (0.0, None), (1.0, 1.7)):
        check(dtype, kind, 4, 2, 128, 16, 200, after(200, [(100, 1), (37, 1)]), seed=12, std=std, scale=scale)
        check(dtype, kind, 4, 2, 64, 16, 200, after(200, [(77, 40), (3, 3)]), seed=13, std=std, scale=scale)


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_the_same_as_without_sharing(dtype, kind):
    """One oracle for both calls: what kv_cache_attend gives for rows that hold the prefix's pages."""
    b = Batch(dtype, kind, 2, 64, 16, 96, after(96, [(40, 1), (3, 1), (200, 1)]), 14)
    q = tokens(b, 8, 64, 14)
    out, cache = torch.empty_like(q).cuda(), b.handle()
    size, call = (B.kv8_cache_attend_workspace_size, B.kv8_cache_attend) if kind == "e4m3" else (B.kv_cache_attend_workspace_size, B.kv_cache_attend)
    ws = B.workspace(size(cache, 3, 3, 8, 1, 300))
    call(cache, q.cuda(), b.table.cuda(), i32(b.cu), i32(b.lens), out, ws, 1, 300)
    for got in (out, b.run(q)):
        for sl, want, bound in b.oracle(q):
            within(got[sl], want, bound, f"tokens {sl.start}..{sl.stop}")


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("n", [1, 9, 40])
def test_values_that_are_not_finite(dtype, kind, n):
    """In the prefix every token that uses it sees them; behind it only the tokens after them."""
    shared, dh = 80, 128
    reqs = after(shared, [(60, n), (45, n)]) + [(shared, min(n, 9))]  # the last reads its own row
    b = Batch(dtype, kind, 2, dh, 16, shared, reqs, 15)
    q = tokens(b, 8, dh, 15)
    clean = b.run(q)
    bad = shared + 60 - n // 2 - 1  # a key of the first request's new tokens
    page, off = int(b.table[0, bad // 16]), bad % 16

    def spoil(page, off):
        if kind == "e4m3":
            b.cache.vc.view(torch.uint8)[page, 1, off, 7] = 127
        else:
            b.v[page, 1, off, 7] = float("inf")

    def spoilt(got):
        return torch.isnan(got).all() if kind == "e4m3" else (got == float("inf")).all()

    spoil(page, off)
    out = b.run(q)
    same = torch.ones(out.shape, dtype=torch.bool, device="cuda")
    same[bad - (shared + 60 - n):n, 4:, 7] = False
    assert torch.equal(out[same], clean[same]) and spoilt(out[~same])
    spoil(int(b.prefix[2]), 5)
    out = b.run(q)
    same[: 2 * n, 4:, 7] = False
    assert torch.equal(out[same], clean[same]) and spoilt(out[~same])


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_bounds_that_are_too_small(dtype, kind):
    """A prefix that counts as max_shared, lengths that end at their bounds, tokens past max_new."""
    shared, reqs = 64, after(64, [(100, 5), (30, 20)])
    b = Batch(dtype, kind, 2, 128, 16, shared, reqs, 16)
    q = tokens(b, 4, 128, 16)
    say(f"[shared] bounds, {dtype} {kind}")
    out = b.run(q, max_new=3)
    for sl, want, bound in b.oracle(q):
        within(out[sl][:3], want[:3], bound[:3], "computed tokens")
        assert torch.isnan(out[sl][3:]).all()
    out = b.run(q, max_own=50)
    for sl, want, bound in b.oracle(q, lens=[shared + 50, shared + 30]):
        within(out[sl], want, bound, "cut 50 after the prefix")
    b.shared = 10 ** 9  # the device's word says more than the bound
    out = b.run(q, max_shared=shared, max_own=100)
    b.shared = shared
    for sl, want, bound in b.oracle(q):
        within(out[sl], want, bound, "the prefix ends at max_shared")
    b.shared = -7
    out = b.run(q, max_shared=0, max_own=200)
    b.shared = shared
    for sl, want, bound in b.oracle(q):
        within(out[sl], want, bound, "no prefix: all from the rows")


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("more", [0, 40])
def test_offsets_that_descend_stay_in_bounds(dtype, kind, more):
    """The prefix is attended to by the tokens from cu[0] on: those before it, which offsets that
    descend name, get something from within the parts, the others their own."""
    shared, n = 700, 2 + more
    b = Batch(dtype, kind, 2, 64, 16, shared, after(shared, [(20, 0), (30 + n, n), (40 + n, 2 * n)]), 3)
    b.cu = [2 * n, 0, n, 3 * n]
    q = tokens(b, 8, 64, 3)
    out = b.run(q)
    (_, want, bound), = attend_oracle(q, b.k, b.v, b.table[2:], b.cu[2:], b.lens[2:], 0, 64 ** -0.5)
    within(out[2 * n:], want[n:], bound[n:], "the tokens behind cu[0]")


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_prefix_pages_out_of_range_stay_in_the_cache(dtype, kind):
    b = Batch(dtype, kind, 2, 64, 16, 64, after(64, [(20, 1), (9, 1)]), 17)
    if kind == "e4m3":
        for x in (b.cache.kc, b.cache.vc):
            x.view(torch.uint8)[x.view(torch.uint8) % 128 == 127] = 3
        b.cache.kb[:], b.cache.vb[:] = 119, 120
    else:
        b.k, b.v = torch.nan_to_num(b.k), torch.nan_to_num(b.v)
    q = tokens(b, 4, 64, 17)
    b.prefix[1], b.prefix[2] = -3, 2 ** 30
    out = b.run(q)
    b.prefix[1], b.prefix[2] = 0, b.k.shape[0] - 1
    assert torch.equal(out, b.run(q))
    # fewer prefix pages than the shared tokens need: the prefix ends with them
    b.prefix = b.prefix[:3]
    b.shared = 10 ** 6
    out = b.run(q, max_shared=200, max_own=40)
    b.shared = 48
    assert torch.equal(out, b.run(q, max_shared=200, max_own=40))


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_groups_with_prefixes_of_their_own(dtype, kind):
    """Two calls over parts of one step: rows of table, cu + r0 (offsets into all tokens) and kv_len."""
    first, second = Batch(dtype, kind, 2, 64, 16, 64, after(64, [(20, 2), (9, 1)]), 18), Batch(dtype, kind, 2, 64, 16, 150, after(150, [(7, 3), (33, 1), (5, 5)]), 19)
    q = torch.cat([tokens(first, 4, 64, 18), tokens(second, 4, 64, 19)])
    out = torch.full(q.shape, float("nan"), dtype=dtype, device="cuda")
    off = first.cu[-1]
    cu = i32(first.cu + [off + c for c in second.cu[1:]])
    for b, r0 in ((first, 0), (second, 2)):
        call, size = b.calls()
        cache, R = b.handle(), len(b.lens)
        ws = B.workspace(size(cache, R, q.shape[0], 4, max(b.news), b.shared, b.own))
        call(cache, q.cuda(), b.prefix.cuda(), i32([b.shared]), b.table.cuda(), cu[r0:r0 + R + 1], i32(b.lens), out, ws, max(b.news), b.shared, b.own)
    torch.cuda.synchronize()
    for b, o in ((first, 0), (second, off)):
        for sl, want, bound in b.oracle(q[o:o + b.cu[-1]]):
            within(out[o + sl.start:o + sl.stop], want, bound, f"tokens {sl.start}..{sl.stop}")


def test_on_another_stream():
    b = Batch(BF, "e4m3", 2, 128, 16, 300, after(300, [(40, 1), (3, 3)]), 20)
    q = tokens(b, 8, 128, 20)
    here = b.run(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert torch.equal(here, b.run(q, stream=s))


@pytest.mark.parametrize("seed", range(40))
def test_drawn(seed):
    rng = random.Random(seed)
    h_q, h_kv = rng.choice([(4, 4), (8, 2), (7, 1), (28, 4), (16, 1), (12, 4), (3, 3)])
    shared = rng.choice([0, rng.randint(1, 60), rng.randint(1, 1500), rng.randint(1, 4000)])
    reqs = []
    for _ in range(rng.randint(1, 12)):
        n = rng.choice([0, 1, 1, rng.randint(1, 16), rng.randint(1, 100)])
        past = shared + rng.choice([0, rng.randint(0, 40), rng.randint(0, 900)]) if rng.random() < 0.85 else rng.randint(0, shared)
        reqs.append((past + n, n))
    if not sum(n for _, n in reqs):
        reqs.append((shared + 17, 1))
    dtype, kind = rng.choice(KINDS)
    check(dtype, kind, h_q, h_kv, rng.choice([64, 128]), rng.choice([16, 32, 64, 128, 256]), shared, reqs, seed=seed, apart=rng.random() < 0.5,
          strided=rng.random() < 0.3, pad=rng.choice([0, 0, 3]))


# ---- together ------------------------------------------------------------------------


@pytest.mark.parametrize("graphed", [False, True])
@pytest.mark.parametrize("dtype,kind", KINDS)
def test_steps_of_a_batch_behind_one_prompt(graphed, dtype, kind):
    """A prompt is written once; then requests with its pages in their rows are planned, written
    and attended to step by step, dropping tokens but never the prompt's, one of them starting
    over. In a graph, one capture serves every step, with eager work between the replays."""
    g = torch.Generator().manual_seed(21)
    R, h_q, h_kv, dh, page, n_pages, cols, cap, shared = 3, 8, 2, 64, 16, 32, 12, 64, 48
    shape = (n_pages, h_kv, page, dh)
    if kind == "e4m3":
        junk = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8).cuda()  # noqa: E731
        cache = B.KVCache8(junk(*shape).view(E4M3), junk(*shape).view(E4M3), junk(*shape[:3]), junk(*shape[:3]), dtype)
        append, attend, size = B.kv8_cache_append, B.kv8_cache_attend_shared, B.kv8_cache_attend_shared_workspace_size
        held_kv = lambda: [values(c.cpu(), b.cpu()) for c, b in ((cache.k, cache.k_exp), (cache.v, cache.v_exp))]  # noqa: E731
    else:
        cache = B.KVCache(*(torch.full(shape, float("nan"), dtype=dtype, device="cuda") for _ in range(2)))
        append, attend, size = B.kv_cache_append, B.kv_cache_attend_shared, B.kv_cache_attend_shared_workspace_size
        held_kv = lambda: [cache.k.cpu().float(), cache.v.cpu().float()]  # noqa: E731
    ang = torch.arange(200)[:, None] * 10000.0 ** (-torch.arange(0, dh, 2) / dh)[None]
    rope = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous().cuda()
    prefix = i32([5, 9, 2])
    table = torch.full((R, cols), -1, dtype=torch.int32, device="cuda")
    table[:, :3] = prefix
    free = [p for p in range(n_pages) if p not in (5, 9, 2)]
    st = dict(held=i32([shared] * R), ctx=i32([shared] * R), new=i32([0] * R), free=i32(free + [-1] * 3), n=i32([len(free)]), n2=i32([0]),
              cu=i32([0] * (R + 1)), kv=i32([0] * R), pos=i32([0] * cap), slot=i32([0] * cap), status=i32([9]), shared=i32([shared]))
    # the prompt: planned by hand, written once
    pk, pv = (torch.randn((shared, h_kv, dh), generator=g).to(dtype) for _ in range(2))
    at = i32([int(prefix[p // page]) * page + p % page for p in range(shared)])
    append(cache, pk.cuda(), pv.cuda(), at, q=torch.zeros((shared, h_q, dh), dtype=dtype, device="cuda"),
           q_out=torch.empty((shared, h_q, dh), dtype=dtype, device="cuda"), pos=i32(list(range(shared))), rope=rope)
    qkv = torch.zeros((cap, h_q + 2 * h_kv, dh), dtype=dtype, device="cuda")
    q_rot, out = (torch.zeros((cap, h_q, dh), dtype=dtype, device="cuda") for _ in range(2))
    ws = B.workspace(size(cache, R, cap, h_q, 40, 64, 140))

    def step(stream=None):
        B.kv_cache_plan(cache, st["held"], st["ctx"], st["new"], table, st["free"], st["n"], st["n2"], st["cu"], st["kv"], st["pos"], st["slot"],
                        st["status"], stream=stream)
        append(cache, qkv[:, h_q:h_q + h_kv], qkv[:, h_q + h_kv:], st["slot"], q=qkv[:, :h_q], q_out=q_rot, pos=st["pos"], rope=rope, stream=stream)
        attend(cache, q_rot, prefix, st["shared"], table, st["cu"], st["kv"], out, ws, 40, 64, 140, stream=stream)

    graph = None
    if graphed:
        step()
        torch.cuda.synchronize()
        st["n"].copy_(st["n2"])
        graph, cap_stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=cap_stream):
            step(cap_stream)
    plan = [([0, 0, 0], [20, 7, 1]), ([20, 7, 1], [1, 1, 1]), ([21, 8, 2], [16, 16, 16]), ([24, 19, 2], [1, 1, 1]), ([25, 0, 3], [16, 40, 0]),
            ([30, 33, 3], [1, 1, 1]), ([31, 34, 0], [1, 1, 0]), ([32, 35, 0], [16, 1, 33])]
    held = [0] * R
    for n, (ctx, new) in enumerate(plan):
        say(f"[shared steps] {dtype} {kind} graph={graphed} step {n}: keep {ctx}, new {new}")
        T = sum(new)
        qkv[:T] = torch.randn((T, h_q + 2 * h_kv, dh), generator=g).to(dtype).cuda()
        st["held"].copy_(i32([shared + h for h in held])), st["ctx"].copy_(i32([shared + c for c in ctx])), st["new"].copy_(i32(new))
        out.fill_(float("nan"))
        graph.replay() if graphed else step()
        torch.cuda.synchronize()
        assert st["status"].item() == 0
        st["n"].copy_(st["n2"])
        k, v = held_kv()
        t = 0
        for r in range(R):
            m = shared + ctx[r] + new[r]
            if new[r]:
                kk, vv = (rows_of(x, table[r].cpu(), m) for x in (k, v))
                lo, hi = S.seen(m, new[r], 0)
                want, spread, reach = S.attend(f64(q_rot[t:t + new[r]]), f64(kk), f64(vv), lo, hi, dh ** -0.5)
                within(out[t:t + new[r]], want, attend_bound(want, spread, reach, m, dh, dtype), f"step {n} request {r}")
            t += new[r]
        assert torch.isnan(out[T:]).all()
        held = [c + x for c, x in zip(ctx, new)]
        used = sum(-(-(shared + h) // page) - 3 for h in held)
        assert st["n"].item() == n_pages - 3 - used
    # the prompt's tokens are as they were written
    vv = rows_of(held_kv()[1], table[0].cpu(), shared)
    assert np.array_equal(f64(vv), S.stand_for(*S.quantise(f64(pv))) if kind == "e4m3" else f64(pv))
