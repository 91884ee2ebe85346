"""Argument checks of the 8-bit cache and of attention over a shared prefix on the CPU: every
refusal happens before any HIP call, with the documented status; sizes of workspaces."""

import ctypes
import random

import pytest
import torch

try:
    from contextual_activation_sparsity_amd import binding as B
except ImportError:  # library not built
    B = None

pytestmark = [pytest.mark.skipif(B is None, reason="libsparse_ffn.so not built"), pytest.mark.filterwarnings("ignore")]

FAKE = 0x100000  # 256-aligned fake device address; never dereferenced on these paths


def _kv(n_pages=100, page=16, h_kv=8, dh=128, dtype=1, reserved=0, k=FAKE, v=FAKE):
    return B.sfn_kv(n_pages, page, h_kv, dh, dtype, reserved, k, v)


def _kv8(k_exp=FAKE, v_exp=FAKE, **kw):
    return B.sfn_kv8(_kv(**kw), k_exp, v_exp)


def append(kv=None, **kw):
    a = dict(T=3, h_q=32, q=FAKE, qs=6272, k=FAKE, ks=6272, v=FAKE, vs=6272, pos=FAKE, slot=FAKE, rope=FAKE, n_pos=64, rot=128, q_out=FAKE)
    a.update(kw)
    return B.raw().kv8_cache_append(kv or _kv8(), *a.values(), None)


def read(kv=None, **kw):
    a = dict(T=3, slot=FAKE, k=FAKE, ks=1024, v=FAKE, vs=1024)
    a.update(kw)
    return B.raw().kv8_cache_read(kv or _kv8(), *a.values(), None)


def attend(kv=None, **kw):
    a = dict(R=2, T=3, h_q=32, q=FAKE, qs=4096, table=FAKE, max_pages=50, cu=FAKE, kv_len=FAKE, max_new=2, max_len=700, scale=0.1, window=0,
             out=FAKE, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return B.raw().kv8_cache_attend(kv or _kv8(), *a.values(), None)


def shared(kv=None, **kw):
    a = dict(R=2, T=3, h_q=32, q=FAKE, qs=4096, prefix=FAKE, prefix_pages=20, shared_len=FAKE, table=FAKE, max_pages=50, cu=FAKE, kv_len=FAKE,
             max_new=2, max_shared=300, max_own=200, scale=0.1, out=FAKE, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    plain = isinstance(kv, B.sfn_kv)
    return (B.raw().kv_cache_attend_shared if plain else B.raw().kv8_cache_attend_shared)(kv or _kv8(), *a.values(), None)


BAD_CACHES = [
    (dict(n_pages=0), "ESHAPE"), (dict(page=8), "ESHAPE"), (dict(page=48), "ESHAPE"), (dict(n_pages=2 ** 27, page=16), "ESHAPE"), (dict(h_kv=0), "ESHAPE"),
    (dict(h_kv=1025), "ESHAPE"), (dict(dh=96), "ESHAPE"), (dict(dtype=2), "EDTYPE"), (dict(reserved=1), "EINVAL"), (dict(k=FAKE + 8), "EALIGN"),
    (dict(v=FAKE + 2), "EALIGN")]


@pytest.mark.parametrize("bad,status", BAD_CACHES + [(dict(k_exp=FAKE + 4), "EALIGN"), (dict(v_exp=FAKE + 1), "EALIGN")], ids=str)
def test_every_call_checks_the_cache(bad, status):
    want, kv = getattr(B, "SFN_" + status), _kv8(**bad)
    assert append(kv) == want and read(kv) == want and attend(kv) == want and shared(kv) == want
    assert B.raw().kv8_cache_attend_workspace_size(kv, 1, 1, 8, 1, 10) == 0
    assert B.raw().kv8_cache_attend_shared_workspace_size(kv, 1, 1, 8, 1, 10, 10) == 0
    if "k_exp" not in bad and "v_exp" not in bad:
        assert shared(_kv(**bad)) == want and B.raw().kv_cache_attend_shared_workspace_size(_kv(**bad), 1, 1, 8, 1, 10, 10) == 0


@pytest.mark.parametrize("null", ["k", "v", "k_exp", "v_exp"])
def test_null_arrays(null):
    kv = _kv8(**{null: None})
    assert append(kv) == read(kv) == attend(kv) == shared(kv) == B.SFN_EINVAL
    assert B.raw().kv8_cache_attend_workspace_size(kv, 1, 1, 8, 1, 10) > 0  # sizes need the shape alone


def test_null_cache():
    lib = B.raw()
    for call in (lib.kv8_cache_append, lib.kv8_cache_read, lib.kv8_cache_attend, lib.kv8_cache_attend_shared, lib.kv_cache_attend_shared):
        assert call(None, *[0.0 if t is ctypes.c_float else 0 for t in call.argtypes[1:]]) == B.SFN_EINVAL
    for size in (lib.kv8_cache_attend_workspace_size, lib.kv8_cache_attend_shared_workspace_size, lib.kv_cache_attend_shared_workspace_size):
        assert size(None, *[1] * (len(size.argtypes) - 1)) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), "ESHAPE"), (dict(T=262145), "ESHAPE"), (dict(h_q=-1), "ESHAPE"), (dict(h_q=1025), "ESHAPE"), (dict(q=None), "EINVAL"),
    (dict(q_out=None), "EINVAL"), (dict(h_q=0), "EINVAL"), (dict(k=None), "EINVAL"), (dict(v=None), "EINVAL"), (dict(slot=None), "EINVAL"),
    (dict(pos=None), "EINVAL"), (dict(rope=None), "EINVAL"), (dict(rot=0), "ESHAPE"), (dict(rot=24), "ESHAPE"), (dict(rot=144), "ESHAPE"),
    (dict(n_pos=0), "ESHAPE"), (dict(qs=4088), "ESHAPE"), (dict(ks=1016), "ESHAPE"), (dict(vs=-6272), "ESHAPE"), (dict(qs=6276), "EALIGN"),
    (dict(ks=6275), "EALIGN"), (dict(q=FAKE + 8), "EALIGN"), (dict(k=FAKE + 4), "EALIGN"), (dict(q_out=FAKE + 2), "EALIGN"),
    (dict(rope=FAKE + 4), "EALIGN"), (dict(pos=FAKE + 1), "EALIGN"), (dict(slot=FAKE + 2), "EALIGN")], ids=str)
def test_append_refusals(kw, status):
    assert append(**kw) == getattr(B, "SFN_" + status)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), "ESHAPE"), (dict(T=262145), "ESHAPE"), (dict(slot=None), "EINVAL"), (dict(k=None), "EINVAL"), (dict(v=None), "EINVAL"),
    (dict(ks=1016), "ESHAPE"), (dict(vs=-1024), "ESHAPE"), (dict(ks=1028), "EALIGN"), (dict(vs=1025), "EALIGN"), (dict(k=FAKE + 8), "EALIGN"),
    (dict(v=FAKE + 2), "EALIGN"), (dict(slot=FAKE + 2), "EALIGN")], ids=str)
def test_read_refusals(kw, status):
    assert read(**kw) == getattr(B, "SFN_" + status)


ATTEND_REFUSALS = [
    (dict(R=0), "ESHAPE"), (dict(R=4097), "ESHAPE"), (dict(T=-1), "ESHAPE"), (dict(h_q=0), "ESHAPE"), (dict(h_q=12), "ESHAPE"), (dict(h_q=1032), "ESHAPE"),
    (dict(max_new=0), "ESHAPE"), (dict(max_pages=0), "ESHAPE"), (dict(qs=4095), "ESHAPE"), (dict(qs=4100), "EALIGN"), (dict(q=None), "EINVAL"),
    (dict(table=None), "EINVAL"), (dict(cu=None), "EINVAL"), (dict(kv_len=None), "EINVAL"), (dict(out=None), "EINVAL"), (dict(scale=0.0), "EINVAL"),
    (dict(scale=float("nan")), "EINVAL"), (dict(scale=float("inf")), "EINVAL"), (dict(out=FAKE + 8), "EALIGN"), (dict(table=FAKE + 2), "EALIGN"),
    (dict(cu=FAKE + 1), "EALIGN"), (dict(kv_len=FAKE + 3), "EALIGN"), (dict(ws=None), "EWORKSPACE"), (dict(ws_bytes=2047), "EWORKSPACE"),
    (dict(ws=FAKE + 16), "EALIGN")]


@pytest.mark.parametrize("kw,status", ATTEND_REFUSALS + [(dict(max_len=-1), "ESHAPE"), (dict(max_len=2 ** 30 + 1), "ESHAPE"), (dict(window=-1), "EINVAL")], ids=str)
def test_attend_refusals(kw, status):
    assert attend(**kw) == getattr(B, "SFN_" + status)


@pytest.mark.parametrize("kw,status", ATTEND_REFUSALS + [
    (dict(max_shared=-1), "ESHAPE"), (dict(max_own=-1), "ESHAPE"), (dict(max_shared=2 ** 29, max_own=2 ** 29 + 1), "ESHAPE"), (dict(prefix_pages=0), "ESHAPE"),
    (dict(max_shared=2 ** 31 - 1, max_own=2 ** 31 - 1), "ESHAPE"), (dict(prefix=None), "EINVAL"), (dict(shared_len=None), "EINVAL"), (dict(prefix=FAKE + 2), "EALIGN"),
    (dict(shared_len=FAKE + 1), "EALIGN")], ids=str)
def test_shared_refusals(kw, status):
    assert shared(**kw) == getattr(B, "SFN_" + status) and shared(_kv(), **kw) == getattr(B, "SFN_" + status)


def test_shared_launches_past_32_bits_of_threads_are_refused():
    """4096 requests whose bound is 4096 tokens of 64 query heads over 8: 8.4 million row tiles over the
    heads are launched; the same over 32 key heads are too many."""
    big = dict(R=4096, T=262144, max_new=8192, max_shared=100, max_own=300, ws_bytes=1 << 60, ws=FAKE + 16)
    assert shared(_kv8(h_kv=8), h_q=32, qs=4096, **big) == B.SFN_EALIGN  # it gets to the workspace
    assert shared(_kv8(h_kv=32), h_q=128, qs=16384, **big) == B.SFN_ESHAPE


def test_no_tokens_is_no_work():
    assert append(T=0, q=None, k=None, v=None, slot=None) == B.SFN_OK and read(T=0, slot=None, k=None, v=None) == B.SFN_OK
    assert attend(T=0, q=None, out=None) == B.SFN_OK and shared(T=0, q=None, out=None) == B.SFN_OK


@pytest.mark.parametrize("seed", range(300))
def test_a_programs_largest_bounds_are_enough_for_its_smaller_calls(seed):
    rng = random.Random(seed)
    h_kv = rng.choice([1, 2, 4, 8])
    h_q, dtype, e8 = h_kv * rng.choice([1, 2, 4, 7, 8, 16]), rng.choice([0, 1, 1]), rng.random() < 0.5
    kw = dict(n_pages=1000, h_kv=h_kv, dtype=dtype, dh=rng.choice([64, 128]))
    kv, lib = (_kv8(**kw) if e8 else _kv(**kw)), B.raw()
    log = lambda hi: int(hi ** rng.random())  # noqa: E731
    R, new, T = log(300), log(3000), 0
    T = max(1, min(R * new, log(9000)))
    own, pre = log(40000), log(40000)
    for _ in range(20):
        r, t, n, o, p = (max(1, int(x * rng.choice([1, 1, rng.random()]))) for x in (R, T, new, own, pre))
        need = (lib.kv8_cache_attend_shared_workspace_size if e8 else lib.kv_cache_attend_shared_workspace_size)(kv, R, T, h_q, new, pre, own)
        assert shared(kv, R=r, T=t, h_q=h_q, qs=h_q * 128, max_new=n, max_shared=p, max_own=o, max_pages=9999, prefix_pages=9999, ws=FAKE + 16,
                      ws_bytes=need) == B.SFN_EALIGN, (r, t, n, o, p)
        if e8:
            need = lib.kv8_cache_attend_workspace_size(kv, R, T, h_q, new, own)
            assert attend(kv, R=r, T=t, h_q=h_q, qs=h_q * 128, max_new=n, max_len=o, max_pages=9999, window=rng.choice([0, log(9000)]), ws=FAKE + 16,
                          ws_bytes=need) == B.SFN_EALIGN, (r, t, n, o)


# ---- the binding ---------------------------------------------------------------------


def fake_cuda(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def test_handles_refuse_what_does_not_fit():
    from torch._subclasses.fake_tensor import FakeTensorMode

    with FakeTensorMode():
        e4, u8 = torch.float8_e4m3fn, torch.uint8
        k, e = fake_cuda((9, 2, 16, 64), e4), fake_cuda((9, 2, 16), u8)
        for bad, why in [((k, fake_cuda((9, 2, 16, 128), e4), e, e), "float8_e4m3fn"), ((k, fake_cuda((9, 2, 16, 64), u8), e, e), "float8_e4m3fn"),
                         ((k, k, e, fake_cuda((9, 2, 32), u8)), "uint8"), ((k, k, fake_cuda((9, 2, 16), torch.int8), e), "uint8"),
                         ((k, k, e, e, torch.float16), "bfloat16 or float32"), ((k, k, e, e.to("cuda:1")), "one device"), ((k[0], k[0], e, e), "float8_e4m3fn")]:
            with pytest.raises(ValueError, match=why):
                B.KVCache8(*bad)


def test_a_cache_of_the_other_kind_is_refused():
    kv, kv8 = object.__new__(B.KVCache), object.__new__(B.KVCache8)
    kv.dh = kv8.dh = 64
    x = [None] * 12
    for call, handle, n in [(B.kv8_cache_append, kv, 3), (B.kv8_cache_read, kv, 3), (B.kv8_cache_attend, kv, 8), (B.kv8_cache_attend_shared, kv, 11),
                            (B.kv_cache_attend_shared, kv8, 11), (B.kv_cache_append, kv8, 3), (B.kv_cache_attend, kv8, 8)]:
        with pytest.raises(TypeError, match="KVCache8"):
            call(handle, *x[:n], stream=0)


def test_tensors_and_streams_of_another_device_are_refused(monkeypatch):
    from torch._subclasses.fake_tensor import FakeTensorMode

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    stream = type("Stream", (), {"device_index": 1, "cuda_stream": 0})()
    kv8 = object.__new__(B.KVCache8)
    kv8.addr, kv8.device = 1, 0
    with pytest.raises(ValueError, match="the stream is of cuda:1, the current device is cuda:0"):
        B.kv8_cache_read(kv8, None, None, None, stream=stream)
    kv8.device = 1
    with pytest.raises(ValueError, match="the cache is on cuda:1, the current device is cuda:0"):
        B.kv8_cache_read(kv8, None, None, None, stream=0)
    c = _kv8(h_kv=2, dh=64)
    at = ctypes.addressof(c)
    with FakeTensorMode():
        rows = lambda d: torch.empty((4, 2, 64), dtype=torch.bfloat16, device=f"cuda:{d}")  # noqa: E731
        i = lambda d, *s: torch.empty(s or (9,), dtype=torch.int32, device=f"cuda:{d}")  # noqa: E731
        with pytest.raises(ValueError, match="v_out is on cuda:1, the call is for cuda:0"):
            B._args.read8(at, i(0), rows(0), rows(1), 0, 0)
        with pytest.raises(ValueError, match="slot is on cuda:0, the call is for cuda:1"):
            B._args.read8(at, i(0), rows(1), rows(1), 0, 1)
        with pytest.raises(ValueError, match="rope is on cuda:1"):
            B._args.append8(at, rows(0), rows(0), i(0), None, None, i(0), torch.empty((9, 64), device="cuda:1"), 0, 0)
        with pytest.raises(ValueError, match="kv_len is on cuda:1"):
            B._args.attend8(at, rows(0), i(0, 2, 3), i(0), i(1), rows(0), i(0), 1, 9, 0.1, 0, 0, 0)
        with pytest.raises(ValueError, match="prefix is on cuda:1"):
            B._args.attend_shared8(at, rows(0), i(1), i(0), i(0, 2, 3), i(0), i(0), rows(0), i(0), 1, 9, 9, 0.1, 0, 0)
        # the calls that were there before do not ask: the library's own refusal of null addresses
        assert B._args.append(at, rows(0), rows(1), i(0), None, None, None, None, 0) == B.SFN_EINVAL


def test_layouts_are_named():
    from torch._subclasses.fake_tensor import FakeTensorMode

    c = _kv8(h_kv=2, dh=64)
    at = ctypes.addressof(c)
    with FakeTensorMode():
        rows = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        i = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
        good = rows(4, 2, 64)
        for call, why in [
            (lambda: B._args.read8(at, i(3), good, good, 0, 0), "slot holds 3 elements, needs 4"),
            (lambda: B._args.read8(at, i(4), rows(4, 3, 64), good, 0, 0), r"k_out must be \[T, 2, 64\]"),
            (lambda: B._args.read8(at, i(4), good, rows(5, 2, 64), 0, 0), r"v_out must be \[4, 2, 64\]"),
            (lambda: B._args.read8(at, i(4), good, good.float(), 0, 0), "v_out must be BFloat16"),
            (lambda: B._args.append8(at, good.float(), good, i(4), None, None, None, None, 0, 0), "k must be BFloat16"),
            (lambda: B._args.append8(at, good, good, i(4), rows(4, 5, 64), rows(4, 4, 64), None, None, 0, 0), "q_out holds 1024 elements, needs 1280"),
            (lambda: B._args.attend8(at, rows(4, 2, 128), i(2, 3), i(3), i(2), good, i(9), 1, 9, 0.1, 0, 0, 0), r"q must be \[T, heads, 64\]"),
            (lambda: B._args.attend_shared8(at, good, i(3), i(0), i(2, 3), i(3), i(2), good, i(9), 1, 9, 9, 0.1, 0, 0), "shared_len holds 0 elements, needs 1"),
            (lambda: B._args.attend_shared8(at, good, i(3), i(1), i(6), i(3), i(2), good, i(9), 1, 9, 9, 0.1, 0, 0), r"table must be \[R, max_pages\]"),
            (lambda: B._args.attend_shared8(at, good, i(3), i(1), i(2, 3), i(3), i(2), good, i(9), 1, 9, 2 ** 31, 0.1, 0, 0), "max_own is too large"),
        ]:
            with pytest.raises(ValueError, match=why):
                call()
        with pytest.raises(TypeError, match="expected 6 arguments, got 3"):
            B._args.read8(at, i(4), good)
