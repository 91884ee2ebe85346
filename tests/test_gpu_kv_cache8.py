"""The 8-bit key/value cache on the GPU: its append, its read and its attention, against the
float64 oracle."""

import random

import numpy as np
import pytest
import torch

from oracle import serving as S
from tests.cache8_helpers import BF, E4M3, F32, Cache8, random_cache8, values
from tests.helpers import say
from tests.serving_helpers import U32, UB, attend_bound, attend_oracle, f64, rows_of, within

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from contextual_activation_sparsity_amd import binding as B


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def u8(x):
    return x.view(torch.uint8).cpu().numpy()


def rope_table(n_pos, rot):
    ang = torch.arange(n_pos, dtype=torch.float64)[:, None] * (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot))[None]
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


def any_cache(n_pages, h_kv, page, dh, dtype, seed):
    """A cache of any codes and bytes."""
    g = torch.Generator().manual_seed(seed)
    codes = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8).cuda()  # noqa: E731
    shape = (n_pages, h_kv, page)
    return B.KVCache8(codes(*shape, dh).view(E4M3), codes(*shape, dh).view(E4M3), codes(*shape), codes(*shape), dtype)


# ---- read ----------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dh", [64, 128])
def test_read_every_code_with_every_byte(dtype, dh):
    """256 rows, row b with byte b: exact values, those of bytes out of use the nearest byte's."""
    n = 256 * 256 // dh
    codes = torch.arange(256, dtype=torch.uint8).repeat(256).reshape(-1, dh)  # row i: codes (i dh) mod 256 on
    b = (torch.arange(n) // (n // 256)).to(torch.uint8)
    kc = codes.reshape(n // 16, 1, 16, dh).cuda()
    exps = b.reshape(n // 16, 1, 16).cuda()
    cache = B.KVCache8(kc.view(E4M3), kc.flip(-1).contiguous().view(E4M3), exps, exps.clone(), dtype)
    out = torch.zeros((n, 2, dh), dtype=dtype, device="cuda")
    say(f"[read8] every code, {dtype} dh={dh}")
    B.kv8_cache_read(cache, i32(list(range(n))), out[:, :1], out[:, 1:])
    torch.cuda.synchronize()
    want = S.stand_for(codes.numpy(), b.numpy())
    assert np.array_equal(f64(out[:, 0]), want, equal_nan=True)
    assert np.array_equal(f64(out[:, 1]), S.stand_for(codes.flip(-1).numpy(), b.numpy()), equal_nan=True)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,h_kv,dh,page", [(1, 8, 128, 16), (3, 3, 64, 32), (130, 1, 128, 64), (37, 5, 64, 256), (700, 2, 128, 128)])
def test_read_rows_by_slots(dtype, T, h_kv, dh, page):
    """Any order, slots twice and outside the cache, rows of wider ones; nothing else is written."""
    say(f"[read8] {dtype} T={T} h_kv={h_kv} dh={dh} page={page}")
    g = torch.Generator().manual_seed(T)
    n_pages = T // page + 3
    cache = any_cache(n_pages, h_kv, page, dh, dtype, T)
    slot = torch.randint(0, n_pages * page, (T,), generator=g, dtype=torch.int32)
    if T > 2:
        slot[0], slot[2], slot[1] = -1, n_pages * page, slot[T - 1]
    if T > 100:
        slot[77], slot[78] = -(2 ** 31), 2 ** 31 - 1
    rows = torch.full((T, 2 * h_kv + 1, dh), 7.0, dtype=dtype, device="cuda")
    k_out = torch.full((T, h_kv, dh), 7.0, dtype=dtype, device="cuda")
    B.kv8_cache_read(cache, slot.cuda(), k_out, rows[:, 1:h_kv + 1])
    B.kv8_cache_read(cache, slot.cuda()[:0], k_out[:0], rows[:0, :h_kv])
    torch.cuda.synchronize()
    assert (rows[:, 0] == 7.0).all() and (rows[:, h_kv + 1:] == 7.0).all()
    for got, codes, b in ((k_out, cache.k, cache.k_exp), (rows[:, 1:h_kv + 1], cache.v, cache.v_exp)):
        want = S.stand_for(u8(codes), u8(b)).transpose(0, 2, 1, 3).reshape(-1, h_kv, dh)
        inside = (slot >= 0) & (slot < n_pages * page)
        want = np.where(inside.numpy()[:, None, None], want[np.clip(slot.numpy(), 0, n_pages * page - 1)], 0.0)
        assert np.array_equal(f64(got), want, equal_nan=True)


# ---- append --------------------------------------------------------------------------


def check_append(dtype, q, k, v, slot, pos, rope, cache):
    """Runs the append and compares codes, bytes and q with the oracle's; cells without a token
    keep what they held."""
    T, h_kv, dh = k.shape
    n_pages, page = cache.n_pages, cache.page
    rot = rope.shape[1] if rope is not None else 0
    before = [u8(x).copy() for x in (cache.k, cache.v, cache.k_exp, cache.v_exp)]
    q_out = None if q is None else torch.full(q.shape, float("nan"), dtype=dtype, device="cuda")
    B.kv8_cache_append(cache, k, v, slot.cuda(), q=q, q_out=q_out, pos=None if rope is None else pos.cuda(),
                       rope=None if rope is None else rope.cuda())
    torch.cuda.synchronize()
    p = pos.numpy() if rot else np.zeros(T, int)
    tab = rope.numpy() if rot else np.zeros((1, 0))
    if q is not None:
        mag = lambda x: np.abs(x) + np.abs(np.roll(x, rot // 2, -1)) + np.abs(np.roll(x, -(rot // 2), -1))  # noqa: E731
        want = S.rotate(f64(q), p, tab, rot)
        within(q_out, want, UB[dtype] * np.abs(want) + 3 * U32 * mag(f64(q)), "q")
    for x, got_codes, got_b, codes, b, name in ((S.rotate(f64(k), p, tab, rot), cache.k, cache.k_exp, before[0], before[2], "k"),
                                                (f64(v), cache.v, cache.v_exp, before[1], before[3], "v")):
        new_codes, new_b = S.quantise(x)
        at = [t for t in range(T) if 0 <= int(slot[t]) < n_pages * page]
        s = slot.numpy()[at]
        codes[s // page, :, s % page], b[s // page, :, s % page] = new_codes[at], new_b[at]
        assert np.array_equal(u8(got_b), b), name
        got_codes = u8(got_codes)
        assert np.array_equal(got_codes & 127, codes & 127), (name, np.argwhere((got_codes & 127) != (codes & 127))[:5])
        signed = (codes & 127) % 127 != 0  # neither a zero nor NaN
        assert np.array_equal(got_codes[signed], codes[signed]), name


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,h_q,h_kv,dh,page,rot", [
    (1, 32, 8, 128, 16, 128), (3, 7, 7, 64, 32, 64), (37, 28, 4, 128, 64, 64), (5, 0, 3, 64, 16, 32), (9, 4, 2, 128, 256, 48),
    (2, 5, 1, 64, 16, 0), (130, 1, 1, 128, 16, 16), (400, 8, 2, 128, 128, 128), (4, 64, 37, 128, 16, 96)])
def test_append_writes_the_oracles_codes(dtype, T, h_q, h_kv, dh, page, rot):
    say(f"[append8] {dtype} T={T} heads={h_q}/{h_kv} dh={dh} page={page} rot={rot}")
    g = torch.Generator().manual_seed(T * 100 + h_q)
    n_pages = T // page + 3
    size = torch.exp(2 * torch.randn((T, h_q + 2 * h_kv + 1, 1), generator=g))
    qkv = (torch.randn((T, h_q + 2 * h_kv + 1, dh), generator=g) * size).to(dtype).cuda()  # one head more than is used: strided rows
    slot = torch.randperm(n_pages * page, generator=g)[:T].to(torch.int32)
    if T > 2:
        slot[0], slot[2] = -1, n_pages * page  # these write nothing
    pos = torch.randint(-3, 60, (T,), generator=g).to(torch.int32)
    check_append(dtype, qkv[:, :h_q] if h_q else None, qkv[:, h_q:h_q + h_kv], qkv[:, h_q + h_kv:h_q + 2 * h_kv], slot, pos,
                 rope_table(50, rot) if rot else None, any_cache(n_pages, h_kv, page, dh, dtype, 5))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_rows_at_the_ends_of_the_range(dtype):
    """Zeros, the smallest and the largest numbers, powers of two and 448 times them, borders
    between codes, infinities and NaN."""
    say(f"[append8] ends of the range, {dtype}")
    dh, T = 64, 24
    x = torch.zeros((T, 1, dh), dtype=torch.float64)
    ramp = torch.linspace(-1, 1, dh, dtype=torch.float64)
    top = [0.0, 1e-45, 1e-40, 2.0 ** -126, 448 * 2.0 ** -117, 449 * 2.0 ** -117, 1e-30, 448.0, 448 * 2.0 ** 50, 449.0, 450.0, 256.0, 1.0, 1.75,
           1.7578125, 2.0 ** 100, 448 * 2.0 ** 118, 450 * 2.0 ** 118, 448 * 2.0 ** 119, 3.38e38]
    for t, m in enumerate(top):
        x[t, 0] = ramp * m
    x[20, 0, :8] = torch.tensor([448.0, 17.0, 19.0, 2.0 ** -10, 1.5 * 2.0 ** -9, -17.0, -19.0, 3 * 2.0 ** -10])
    x[21, 0, :5] = torch.tensor([float("inf"), 1.0, float("nan"), -float("inf"), -3.0])
    x[22] = float("nan")
    x[23, 0, 3] = -0.0
    x = x.to(dtype).cuda()
    cache = any_cache(4, 1, 16, dh, dtype, 6)
    check_append(dtype, None, x, x.flip(0), torch.arange(3, 3 + T, dtype=torch.int32), torch.zeros(T), None, cache)


def test_append_in_place_and_empty():
    g = torch.Generator().manual_seed(1)
    q = torch.randn((4, 6, 64), generator=g).to(BF).cuda()
    k = torch.randn((4, 2, 64), generator=g).to(BF).cuda()
    cache = any_cache(2, 2, 16, 64, BF, 7)
    rope, pos, slot = rope_table(9, 64).cuda(), i32([1, 2, 3, 8]), i32([0, 1, 2, 3])
    out = torch.empty_like(q)
    B.kv8_cache_append(cache, k, k, slot, q=q, q_out=out, pos=pos, rope=rope)
    B.kv8_cache_append(cache, k, k, slot, q=q, q_out=q, pos=pos, rope=rope)
    B.kv8_cache_append(cache, k[:0], k[:0], slot[:0])
    torch.cuda.synchronize()
    assert torch.equal(q, out)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_what_is_read_can_be_appended_again(dtype):
    """Rows read and appended without rotation are the same rows."""
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn((50, 3, 128), generator=g).to(dtype).cuda() for _ in range(2))
    cache, other = any_cache(5, 3, 16, 128, dtype, 8), any_cache(5, 3, 16, 128, dtype, 9)
    slot, slot2 = (torch.randperm(80, generator=g)[:50].to(torch.int32).cuda() for _ in range(2))
    B.kv8_cache_append(cache, k, v, slot)
    a, b, c, d = (torch.empty_like(k) for _ in range(4))
    B.kv8_cache_read(cache, slot, a, b)
    B.kv8_cache_append(other, a, b, slot2)
    B.kv8_cache_read(other, slot2, c, d)
    torch.cuda.synchronize()
    assert torch.equal(a, c) and torch.equal(b, d)
    assert ((a.float() - k.float()).abs() <= 2.0 ** -4 * k.float().abs() + 2.0 ** -10 * 2.0 ** -6).all()


# ---- attention -----------------------------------------------------------------------


def run_attend(cache, q, table, cu, lens, window=0, max_new=None, max_len=None, scale=None, strided=False, stream=None):
    R, (T, h_q, dh) = len(lens), q.shape
    max_new = max(1, max(b - a for a, b in zip(cu, cu[1:]))) if max_new is None else max_new
    max_len = max(lens) if max_len is None else max_len
    qd = q.cuda()
    if strided:
        wide = torch.full((T, h_q + 3, dh), float("nan"), dtype=q.dtype, device="cuda")
        wide[:, 1:h_q + 1] = qd
        qd = wide[:, 1:h_q + 1]
    out = torch.full((T, h_q, dh), float("nan"), dtype=q.dtype, device="cuda")
    handle = cache.on_gpu(B, q.dtype)
    ws = B.workspace(B.kv8_cache_attend_workspace_size(handle, R, T, h_q, max_new, max_len))
    ws[2048:] = 255  # scratch is NaN: what is not written must not be read
    args = (handle, qd, table.cuda(), i32(cu), i32(lens), out, ws, max_new, max_len)
    B.kv8_cache_attend(*args, scale=scale, window=window, stream=stream)
    torch.cuda.synchronize()
    first = out.clone()
    B.kv8_cache_attend(*args, scale=scale, window=window, stream=stream)
    torch.cuda.synchronize()
    as_bits = torch.int16 if q.dtype == BF else torch.int32
    assert torch.equal(first.view(as_bits), out.view(as_bits)), "two runs differ"
    assert int(ws[:2048].to(torch.int32).sum()) == 0
    return out


def cu_of(news):
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    return cu


def check_attend(dtype, h_q, h_kv, dh, page, reqs, window=0, seed=0, scale=None, std=1.0, **kw):
    """reqs: (kv_len, new tokens) of each request."""
    lens, cu = [r[0] for r in reqs], cu_of(r[1] for r in reqs)
    cache, table = random_cache8(lens, h_kv, dh, page, seed)
    q = (torch.randn((cu[-1], h_q, dh), generator=torch.Generator().manual_seed(seed + 1)) * std).to(dtype)
    say(f"[attend8] {dtype} heads={h_q}/{h_kv} dh={dh} page={page} window={window} reqs={reqs[:6]}")
    out = run_attend(cache, q, table, cu, lens, window, scale=scale, **kw)
    sc = dh ** -0.5 if scale is None else scale
    for sl, want, bound in attend_oracle(q, cache.k, cache.v, table, cu, lens, window, sc):
        within(out[sl], want, bound, f"tokens {sl.start}..{sl.stop}")


HEADS = [(4, 4), (8, 2), (7, 1), (28, 4), (16, 1)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("h_q,h_kv", HEADS)
def test_attend_single_tokens_at_every_edge(dtype, dh, h_q, h_kv):
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 700]
    for page in (16, 64, 256):
        check_attend(dtype, h_q, h_kv, dh, page, [(n, 1) for n in lens], seed=page)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("h_q,h_kv", HEADS)
def test_attend_chunks(dtype, dh, h_q, h_kv):
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
    check_attend(dtype, h_q, h_kv, 128, 16, [(2, 5), (0, 3), (1, 20), (40, 40), (0, 1)], seed=6)
    check_attend(dtype, h_q, h_kv, 64, 32, [(0, 1)], seed=7, max_len=0)
    check_attend(dtype, h_q, h_kv, 64, 32, [(0, 1), (0, 200)], seed=7, max_len=512, window=3)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [1, 4, 16])
def test_attend_long_and_split(dtype, n):
    check_attend(dtype, 4, 1, 128, 64, [(9000, n), (20, n), (4097, n)], seed=8)
    check_attend(dtype, 2, 2, 64, 16, [(6001, n)], seed=9, window=3500)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_sharp_and_flat_scores(dtype):
    check_attend(dtype, 4, 2, 128, 16, [(300, 1), (77, 40)], seed=10, std=60.0)
    check_attend(dtype, 4, 2, 64, 16, [(300, 1), (77, 40)], seed=11, std=0.0)
    check_attend(dtype, 4, 2, 64, 16, [(300, 1), (77, 40)], seed=12, scale=1.7)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("h_q,h_kv,n", [(2, 2, 8), (8, 2, 16), (6, 1, 100)])
def test_attend_tokens_do_not_see_later_nan(dtype, h_q, h_kv, n):
    """A NaN key or value of one token leaves every earlier token's result as it was."""
    lens, cu, dh = [200], [0, n], 128
    cache, table = random_cache8(lens, h_kv, dh, 16, 13)
    q = torch.randn((n, h_q, dh), generator=torch.Generator().manual_seed(14)).to(dtype)
    say(f"[attend8] NaN, {dtype} {h_q}/{h_kv} n={n}")
    clean = run_attend(cache, q, table, cu, lens)
    bad = n // 2  # the token whose value is spoilt
    p = 200 - n + bad
    page, off = int(table[0, p // 16]), p % 16
    vc, kc = cache.vc.view(torch.uint8), cache.kc.view(torch.uint8)
    vc[page, :, off, 3], vc[page, :, off, 64] = 127, 255
    was = kc[page, :, off, 5].clone()
    kc[page, :, off, 5] = 127
    out = run_attend(cache, q, table, cu, lens)
    assert torch.equal(out[:bad], clean[:bad])
    assert torch.isnan(out[bad:]).all()
    kc[page, :, off, 5] = was
    out = run_attend(cache, q, table, cu, lens)
    keep = [d for d in range(dh) if d not in (3, 64)]
    assert torch.equal(out[:bad], clean[:bad])
    assert torch.equal(out[bad:][..., keep], clean[bad:][..., keep])
    assert torch.isnan(out[bad:][..., [3, 64]]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_rows_of_very_different_sizes(dtype):
    """Values of 2^100 under no weight, of 2^-100 under all of it, and rows of zeros."""
    lens, cu, dh = [150, 70], [0, 1, 41], 64
    cache, table = random_cache8(lens, 2, dh, 16, 15, spread=0.0)
    for r, n in enumerate(lens):
        for p in range(n):
            page, off = int(table[r, p // 16]), p % 16
            cache.vb[page, :, off] = 227 if p % 7 == 3 else 27 if p % 7 == 5 else int(cache.vb[page, 0, off])
            if p % 7 == 3:  # keys that no query likes: -64 in a direction that all queries have
                cache.kc.view(torch.uint8)[page, :, off] = 0
                cache.kc.view(torch.uint8)[page, :, off, 0], cache.kb[page, :, off] = 0xfe, 127 + 5
            if p % 11 == 8:
                cache.vc.view(torch.uint8)[page, :, off] = 0
    cache.refresh()
    q = torch.randn((41, 4, dh), generator=torch.Generator().manual_seed(16))
    q[..., 0] = 1.0
    q = q.to(dtype)
    say(f"[attend8] rows of very different sizes, {dtype}")
    out = run_attend(cache, q, table, cu, lens)
    for sl, want, bound in attend_oracle(q, cache.k, cache.v, table, cu, lens, 0, dh ** -0.5):
        within(out[sl], want, bound, f"tokens {sl.start}..{sl.stop}")


@pytest.mark.parametrize("sizes", ["any", "alike"])
def test_attend_pages_out_of_range_stay_in_the_cache(sizes):
    """Rows of any size make scores that are not finite, and NaN; the same ones, bit by bit."""
    cache, table = random_cache8([100], 2, 64, 16, 15)
    table[0, 1], table[0, 2] = -3, 2 ** 30
    for x in (cache.kc, cache.vc):  # pages whose every cell holds a number
        x.view(torch.uint8)[x.view(torch.uint8) % 128 == 127] = 3
    if sizes == "alike":
        cache.kb[:], cache.vb[:] = 119, 120
    q = torch.randn((1, 4, 64)).to(BF)
    out = run_attend(cache, q, table, [0, 1], [100])
    fixed = table.clone()
    fixed[0, 1], fixed[0, 2] = 0, cache.kc.shape[0] - 1
    assert torch.equal(out.view(torch.int16), run_attend(cache, q, fixed, [0, 1], [100]).view(torch.int16))
    assert sizes == "any" or (torch.isfinite(out).all() and (out != 0).all())


def test_offsets_past_32_bits():
    """A cache of 5 GB a side whose pages lie at its end: append, read and attention."""
    h_kv, page, dh, n_pages = 8, 64, 128, 80000
    k = torch.empty((n_pages, h_kv, page, dh), dtype=E4M3, device="cuda")
    v, kb, vb = torch.empty_like(k), *(torch.empty((n_pages, h_kv, page), dtype=torch.uint8, device="cuda") for _ in range(2))
    assert k.numel() > 2 ** 32
    cache = B.KVCache8(k, v, kb, vb, BF)
    g = torch.Generator().manual_seed(16)
    pages = [79999, 0, 79990, 40000]
    kn, vn = (torch.randn((256, h_kv, dh), generator=g).to(BF) for _ in range(2))
    slot = i32([pages[i // 64] * page + i % 64 for i in range(256)])
    say("[cache8] offsets past 32 bits")
    B.kv8_cache_append(cache, kn.cuda(), vn.cuda(), slot)
    a, b = torch.empty((256, h_kv, dh), dtype=BF, device="cuda"), torch.empty((256, h_kv, dh), dtype=BF, device="cuda")
    B.kv8_cache_read(cache, slot, a, b)
    torch.cuda.synchronize()
    for got, x in ((a, kn), (b, vn)):
        assert np.array_equal(f64(got), S.stand_for(*S.quantise(f64(x))))
    small_k, small_v = (x.cpu().reshape(4, 64, h_kv, dh).transpose(1, 2).contiguous() for x in (a, b))
    q = torch.randn((20, 16, dh), generator=g).to(BF)
    for n in (1, 20):
        out = torch.empty((n, 16, dh), dtype=BF, device="cuda")
        ws = B.workspace(B.kv8_cache_attend_workspace_size(cache, 1, n, 16, n, 256))
        B.kv8_cache_attend(cache, q[-n:].cuda(), i32([pages]), i32([0, n]), i32([256]), out, ws, n, 256)
        torch.cuda.synchronize()
        table = torch.arange(4, dtype=torch.int32)[None]
        for _, want, bound in attend_oracle(q[-n:], small_k, small_v, table, [0, n], [256], 0, dh ** -0.5):
            within(out, want, bound, "long cache")


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("window", [0, 130])
def test_attend_prompts_that_fill_the_chip(dh, window):
    """More than 256 row tiles of 128: one group of waves to a workgroup, no splits."""
    check_attend(BF, 16, 16, dh, 32, [(700, 650), (640, 640), (300, 129), (650, 650)], window=window, seed=20)


@pytest.mark.parametrize("R", [1, 3])
def test_attend_nan_among_many_row_tiles(R):
    lens, cu = [650] * R, [650 * r for r in range(R + 1)]
    cache, table = random_cache8(lens, 16, 64, 64, 21)
    q = torch.randn((650 * R, 16, 64), generator=torch.Generator().manual_seed(22)).to(BF)
    say(f"[attend8] NaN among many row tiles R={R}")
    clean = run_attend(cache, q, table, cu, lens)
    p = 300  # of the first request
    cache.vc.view(torch.uint8)[int(table[0, p // 64]), 5, p % 64, 9] = 255
    out = run_attend(cache, q, table, cu, lens)
    same = torch.ones(out.shape, dtype=torch.bool, device="cuda")
    same[p:650, 5, 9] = False
    assert torch.equal(out[same], clean[same]) and torch.isnan(out[~same]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [4, 16])
def test_attend_many_rows_with_splits(dtype, n):
    check_attend(dtype, 8, 2, 128, 64, [(2100, n), (1500, n), (60, n), (900, n)] * (4 if n == 4 else 1) + [(800, n)], seed=23)
    check_attend(dtype, 16, 4, 64, 16, [(1300, n), (1, 1), (777, n), (0, 0), (1024, n)], seed=24, window=900)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [1, 9])
def test_attend_unsplit_items_past_the_chip(dtype, n):
    rng = random.Random(n)
    reqs = [(m + rng.choice([0, 1, rng.randint(0, 340)]), m) for m in (rng.choice([0, 1, n, n]) for _ in range(70))]
    check_attend(dtype, 8, 4, 64, 16, reqs, seed=27)
    check_attend(dtype, 10, 5, 128, 64, reqs, seed=28, window=100)


def test_attend_bounds_that_are_too_small():
    lens, cu = [90, 200], [0, 40, 60]
    for dtype, max_new in ((BF, 3), (F32, 9), (BF, 17)):
        cache, table = random_cache8(lens, 2, 128, 16, 25)
        q = torch.randn((60, 4, 128), generator=torch.Generator().manual_seed(26)).to(dtype)
        say(f"[attend8] max_new {max_new} of 40 and 20, {dtype}")
        out = run_attend(cache, q, table, cu, lens, max_new=max_new)
        for sl, want, bound in attend_oracle(q, cache.k, cache.v, table, cu, lens, 0, 128 ** -0.5):
            within(out[sl][:max_new], want[:max_new], bound[:max_new], "computed tokens")
            assert torch.isnan(out[sl][max_new:]).all()
    out = run_attend(cache, q, table, cu, lens, max_len=100)
    for sl, want, bound in attend_oracle(q, cache.k, cache.v, table, cu, [90, 100], 0, 128 ** -0.5):
        within(out[sl], want, bound, "cut at 100 keys")


def test_attend_on_another_stream():
    lens, cu = [300, 40], [0, 1, 17]
    cache, table = random_cache8(lens, 2, 128, 16, 17)
    q = torch.randn((17, 8, 128)).to(BF)
    here = run_attend(cache, q, table, cu, lens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert torch.equal(here, run_attend(cache, q, table, cu, lens, stream=s))


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


# ---- together ------------------------------------------------------------------------


@pytest.mark.parametrize("graphed", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_steps_with_rollback_over_the_8_bit_cache(graphed, dtype):
    """Prompts, single tokens, a chunk of drafts that the next step drops, and a request that
    ends: plan, append, attention and, at the end, the read. In a graph, one capture serves
    every step; every replay is compared, with eager work between them."""
    g = torch.Generator().manual_seed(18)
    R, h_q, h_kv, dh, page, n_pages, cols, cap = 3, 8, 2, 64, 16, 24, 8, 64
    cache = any_cache(n_pages, h_kv, page, dh, dtype, 19)
    rope = rope_table(200, dh).cuda()
    st = dict(held=i32([0] * R), ctx=i32([0] * R), new=i32([0] * R), table=i32([[-1] * cols] * R), free=i32(list(range(n_pages))),
              n=i32([n_pages]), n2=i32([0]), cu=i32([0] * (R + 1)), kv=i32([0] * R), pos=i32([0] * cap), slot=i32([0] * cap), status=i32([9]))
    qkv = torch.zeros((cap, h_q + 2 * h_kv, dh), dtype=dtype, device="cuda")
    q_rot, out = (torch.zeros((cap, h_q, dh), dtype=dtype, device="cuda") for _ in range(2))
    ws = B.workspace(B.kv8_cache_attend_workspace_size(cache, R, cap, h_q, 48, 128))

    def step(stream=None):
        B.kv_cache_plan(cache, st["held"], st["ctx"], st["new"], st["table"], st["free"], st["n"], st["n2"], st["cu"], st["kv"],
                        st["pos"], st["slot"], st["status"], stream=stream)
        B.kv8_cache_append(cache, qkv[:, h_q:h_q + h_kv], qkv[:, h_q + h_kv:], st["slot"], q=qkv[:, :h_q], q_out=q_rot, pos=st["pos"],
                           rope=rope, stream=stream)
        B.kv8_cache_attend(cache, q_rot, st["table"], st["cu"], st["kv"], out, ws, 48, 128, stream=stream)

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
        say(f"[steps8] {dtype} graph={graphed} step {n}: keep {ctx}, new {new}")
        T = sum(new)
        qkv[:T] = torch.randn((T, h_q + 2 * h_kv, dh), generator=g).to(dtype).cuda()
        st["held"].copy_(i32(held)), st["ctx"].copy_(i32(ctx)), st["new"].copy_(i32(new))
        out.fill_(float("nan"))
        graph.replay() if graphed else step()
        torch.cuda.synchronize()
        assert st["status"].item() == 0
        st["n"].copy_(st["n2"])
        host, t = qkv[:T].cpu(), 0
        k, v = (values(c.cpu(), b.cpu()) for c, b in ((cache.k, cache.k_exp), (cache.v, cache.v_exp)))
        for r in range(R):
            seqs[r] = seqs[r][:ctx[r]] + [(host[t + i, h_q:h_q + h_kv], host[t + i, h_q + h_kv:]) for i in range(new[r])]
            m = len(seqs[r])
            if new[r]:
                kk, vv = (rows_of(x, st["table"][r].cpu(), m) for x in (k, v))
                pure = S.rotate(f64(torch.stack([x[0] for x in seqs[r]])), np.arange(m), rope.cpu().numpy(), dh)
                assert np.array_equal(f64(kk), S.stand_for(*S.quantise(pure)))
                assert np.array_equal(f64(vv), S.stand_for(*S.quantise(f64(torch.stack([x[1] for x in seqs[r]])))))
                lo, hi = S.seen(m, new[r], 0)
                want, spread, reach = S.attend(f64(q_rot[t:t + new[r]]), f64(kk), f64(vv), lo, hi, dh ** -0.5)
                within(out[t:t + new[r]], want, attend_bound(want, spread, reach, m, dh, dtype), f"step {n} request {r}")
            t += new[r]
        assert torch.isnan(out[T:]).all()  # rows behind the last token are left as they were
        held = [c + x for c, x in zip(ctx, new)]
        used = sum(-(-h // page) for h in held)
        assert st["n"].item() == n_pages - used
        at = st["slot"][:max(T, 1)]
        ko, vo = (torch.empty((max(T, 1), h_kv, dh), dtype=dtype, device="cuda") for _ in range(2))
        B.kv8_cache_read(cache, at, ko, vo)
        assert np.array_equal(f64(vo[:T]), S.stand_for(*S.quantise(f64(host[:T, h_q + h_kv:]))))
