"""The paged cache's and the residual norm's argument checks on the CPU: every refusal
happens before any HIP call, with the documented status."""

import ctypes

import pytest

try:
    from contextual_activation_sparsity_amd import binding as B
except ImportError:  # library not built
    B = None

pytestmark = pytest.mark.skipif(B is None, reason="libsparse_ffn.so not built")

FAKE = 0x100000  # 256-aligned fake device address; never dereferenced on these paths


def _kv(n_pages=100, page=16, h_kv=8, dh=128, dtype=1, reserved=0, k=FAKE, v=FAKE):
    return B.sfn_kv(n_pages, page, h_kv, dh, dtype, reserved, k, v)


BAD_CACHES = [
    (dict(n_pages=0), "ESHAPE"), (dict(page=8), "ESHAPE"), (dict(page=512), "ESHAPE"), (dict(page=48), "ESHAPE"), (dict(page=0), "ESHAPE"),
    (dict(page=-16), "ESHAPE"), (dict(n_pages=2 ** 27, page=16), "ESHAPE"), (dict(h_kv=0), "ESHAPE"), (dict(h_kv=1025), "ESHAPE"),
    (dict(dh=96), "ESHAPE"), (dict(dh=0), "ESHAPE"), (dict(dtype=2), "EDTYPE"), (dict(reserved=1), "EINVAL"), (dict(k=FAKE + 8), "EALIGN"),
    (dict(v=FAKE + 2), "EALIGN")]


def plan(kv=None, **kw):
    a = dict(R=4, max_pages=10, max_tokens=32, held=FAKE, ctx=FAKE, new=FAKE, table=FAKE, free=FAKE, n=FAKE, n_out=FAKE + 4, cu=FAKE,
             kv_len=FAKE, pos=FAKE, slot=FAKE, status=FAKE)
    a.update(kw)
    return B.raw().kv_cache_plan(kv or _kv(), *a.values(), None)


def append(kv=None, **kw):
    a = dict(T=3, h_q=32, q=FAKE, qs=6272, k=FAKE, ks=6272, v=FAKE, vs=6272, pos=FAKE, slot=FAKE, rope=FAKE, n_pos=64, rot=128, q_out=FAKE)
    a.update(kw)
    return B.raw().kv_cache_append(kv or _kv(), *a.values(), None)


def attend(kv=None, **kw):
    a = dict(R=2, T=3, h_q=32, q=FAKE, qs=4096, table=FAKE, max_pages=50, cu=FAKE, kv_len=FAKE, max_new=2, max_len=700, scale=0.1, window=0,
             out=FAKE, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return B.raw().kv_cache_attend(kv or _kv(), *a.values(), None)


def norm(n=None, **kw):
    a = dict(T=3, h=FAKE, hd=1, y=FAKE, yd=0, gate=None, gs=0, ho=FAKE, xo=FAKE)
    a.update(kw)
    return B.raw().residual_norm(n or B.sfn_norm(4096, 1, 1e-5, 1.0, FAKE, FAKE), *a.values(), None)


@pytest.mark.parametrize("bad,status", BAD_CACHES, ids=lambda x: str(x))
def test_every_call_checks_the_cache(bad, status):
    want = getattr(B, "SFN_" + status)
    kv = _kv(**bad)
    assert plan(kv) == want and append(kv) == want and attend(kv) == want
    assert B.raw().kv_cache_attend_workspace_size(kv, 1, 1, 8, 1, 10) == 0


def test_null_cache():
    for call, n in ((B.raw().kv_cache_plan, 16), (B.raw().kv_cache_append, 15), (B.raw().kv_cache_attend, 17)):
        assert call(None, *[0.0 if t is ctypes.c_float else 0 for t in call.argtypes[1:]]) == B.SFN_EINVAL
        assert len(call.argtypes) == n + 1
    assert B.raw().kv_cache_attend_workspace_size(None, 1, 1, 8, 1, 10) == 0
    assert append(_kv(k=None)) == B.SFN_EINVAL and attend(_kv(v=None)) == B.SFN_EINVAL


@pytest.mark.parametrize("kw,status", [
    (dict(R=0), "ESHAPE"), (dict(R=4097), "ESHAPE"), (dict(max_tokens=0), "ESHAPE"), (dict(max_tokens=262145), "ESHAPE"),
    (dict(max_pages=0), "ESHAPE"), (dict(R=4096, max_pages=2 ** 20), "ESHAPE"), (dict(max_pages=2 ** 28), "ESHAPE"),
    (dict(n_out=FAKE), "EINVAL")] + [({p: None}, "EINVAL") for p in ("held", "ctx", "new", "table", "free", "n", "n_out", "cu", "kv_len", "pos", "slot", "status")]
    + [({p: FAKE + 2}, "EALIGN") for p in ("held", "ctx", "new", "table", "free", "n", "n_out", "cu", "kv_len", "pos", "slot", "status")], ids=str)
def test_plan_refusals(kw, status):
    assert plan(_kv(k=None, v=None), **kw) == getattr(B, "SFN_" + status)


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
    (dict(R=0), "ESHAPE"), (dict(R=4097), "ESHAPE"), (dict(T=-1), "ESHAPE"), (dict(h_q=0), "ESHAPE"), (dict(h_q=12), "ESHAPE"),
    (dict(h_q=1032), "ESHAPE"), (dict(max_new=0), "ESHAPE"), (dict(max_len=-1), "ESHAPE"), (dict(max_len=2 ** 30 + 1), "ESHAPE"),
    (dict(max_pages=0), "ESHAPE"), (dict(qs=4095), "ESHAPE"), (dict(qs=4100), "EALIGN"), (dict(q=None), "EINVAL"), (dict(table=None), "EINVAL"),
    (dict(cu=None), "EINVAL"), (dict(kv_len=None), "EINVAL"), (dict(out=None), "EINVAL"), (dict(scale=0.0), "EINVAL"), (dict(scale=-1.0), "EINVAL"),
    (dict(scale=float("nan")), "EINVAL"), (dict(scale=float("inf")), "EINVAL"), (dict(window=-1), "EINVAL"), (dict(out=FAKE + 8), "EALIGN"),
    (dict(table=FAKE + 2), "EALIGN"), (dict(cu=FAKE + 1), "EALIGN"), (dict(kv_len=FAKE + 3), "EALIGN"), (dict(ws=None), "EWORKSPACE"),
    (dict(ws_bytes=2047), "EWORKSPACE"), (dict(ws=FAKE + 16), "EALIGN")], ids=str)
def test_attend_refusals(kw, status):
    assert attend(**kw) == getattr(B, "SFN_" + status)


def test_attend_workspace_covers_its_own_calls():
    """The size query's bytes are enough for every window, and one byte under what a call
    needs is refused (the call itself stops at its workspace check, before any launch)."""
    size = B.raw().kv_cache_attend_workspace_size
    kv = _kv(n_pages=20000)
    for R, T, h_q, new, length in [(1, 1, 32, 1, 100000), (3, 48, 64, 16, 9000), (1, 1, 8, 1, 1), (40, 40, 16, 1, 4321)]:
        need = size(kv, R, T, h_q, new, length)
        assert need >= B.SFN_WORKSPACE_HEADER_BYTES
        assert size(kv, R, T, h_q, new, length // 2) <= need
        if need > B.SFN_WORKSPACE_HEADER_BYTES:
            assert attend(kv, R=R, T=T, h_q=h_q, qs=h_q * 128, max_new=new, max_len=length, max_pages=20000, ws_bytes=B.SFN_WORKSPACE_HEADER_BYTES) == B.SFN_EWORKSPACE
    assert size(kv, 0, 1, 8, 1, 10) == 0 and size(kv, 1, 1, 9, 1, 10) == 0 and size(kv, 1, 1, 8, 0, 10) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), "ESHAPE"), (dict(hd=2), "EDTYPE"), (dict(yd=-1), "EDTYPE"), (dict(h=None), "EINVAL"), (dict(ho=None, xo=None), "EINVAL"),
    (dict(y=None), "EINVAL"), (dict(y=None, ho=None, gate=FAKE), "EINVAL"), (dict(gate=FAKE, gs=8), "ESHAPE"), (dict(gate=FAKE, gs=4100), "EALIGN"),
    (dict(h=FAKE + 8), "EALIGN"), (dict(y=FAKE + 4), "EALIGN"), (dict(gate=FAKE + 2), "EALIGN"), (dict(ho=FAKE + 8), "EALIGN"), (dict(xo=FAKE + 8), "EALIGN")], ids=str)
def test_norm_refusals(kw, status):
    assert norm(**kw) == getattr(B, "SFN_" + status)


def test_norm_weight_refusals():
    n = lambda d=4096, w=1, eps=1e-5, scale=1.0, post=FAKE, pre=FAKE: B.sfn_norm(d, w, eps, scale, post, pre)  # noqa: E731
    nan, inf = float("nan"), float("inf")
    for m, status in [(n(d=0), "ESHAPE"), (n(d=16392), "ESHAPE"), (n(d=4100), "EALIGN"), (n(w=3), "EDTYPE"), (n(eps=-1.0), "EINVAL"), (n(eps=nan), "EINVAL"),
                      (n(eps=inf), "EINVAL"), (n(scale=nan), "EINVAL"), (n(scale=inf), "EINVAL"), (n(pre=None), "EINVAL"), (n(post=FAKE + 8), "EALIGN"),
                      (n(pre=FAKE + 2), "EALIGN")]:
        assert norm(m) == getattr(B, "SFN_" + status)
    assert B.raw().residual_norm(None, 1, FAKE, 0, FAKE, 0, None, 0, FAKE, FAKE, None) == B.SFN_EINVAL


def test_no_tokens_is_no_work():
    """T = 0 returns success without a launch (there is no GPU here), null addresses allowed."""
    assert append(T=0, q=None, k=None, v=None, slot=None) == B.SFN_OK
    assert attend(T=0, q=None, out=None) == B.SFN_OK
    assert norm(T=0, h=None) == B.SFN_OK
