"""The residual update with its two norms on the GPU, against the float64 oracle."""

import numpy as np
import pytest
import torch

from oracle import serving as S
from tests.helpers import say
from tests.serving_helpers import LAMBDA, U32, UB, f64, within

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from contextual_activation_sparsity_amd import binding as B

BF, F32 = torch.bfloat16, torch.float32


def bounds(h, y, w_pre, w_post, gate, scale, d, hd, wd):
    """h: a few fp32 roundings of the added term (its norm's mean errs by LAMBDA u sqrt(d) / 2
    relative, halved by the root) and of the sum, then the type's. x: the same error of h
    through the norm (its own, and the mean's), a few roundings, then the type's."""
    H, X = S.residual_norm(h, y, w_pre, w_post, gate, scale)
    term = np.abs(H - h)
    fp = U32 * (LAMBDA * np.sqrt(d) + 16.0)
    dh = fp * term + 2 * U32 * np.abs(H)
    r = np.sqrt((H * H).mean(-1, keepdims=True) + 1e-5)
    # the norm of an error vector moves the root by at most its rms
    moved = np.sqrt((dh * dh).mean(-1, keepdims=True)) / r
    dx = (dh / r * np.abs(w_pre) if w_pre is not None else 0.0)
    bx = None if w_pre is None else dx + np.abs(X) * (moved + fp + UB[wd])
    return H, X, dh + UB[hd] * np.abs(H), bx


@pytest.mark.parametrize("h_dt", [BF, F32])
@pytest.mark.parametrize("y_dt", [BF, F32])
@pytest.mark.parametrize("w_dt", [BF, F32])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gated", [0, 1, 2])
def test_residual_norm(h_dt, y_dt, w_dt, post, gated):
    for T, d in [(1, 8), (3, 520), (2, 2048), (1, 4096), (5, 4104), (2, 8192), (3, 11008), (1, 16384), (67, 256)]:
        say(f"[norm] h={h_dt} y={y_dt} w={w_dt} post={post} gate={gated} T={T} d={d}")
        g = torch.Generator().manual_seed(d + T)
        rnd = lambda s, dt, std=1.0: (torch.randn(s, generator=g) * std).to(dt)  # noqa: E731
        h, y = rnd((T, d), h_dt, 2.0), rnd((T, d), y_dt)
        w_pre, w_post = (1 + rnd((d,), w_dt, 0.2)), (1 + rnd((d,), w_dt, 0.2)) if post else None
        gate = None if not gated else rnd((d,) if gated == 1 else (T, d), w_dt)
        cu = lambda t: None if t is None else t.cuda()  # noqa: E731
        norm = B.ResidualNorm(cu(w_pre), w_post=cu(w_post), eps=1e-5, scale=0.5)
        ho, xo = torch.full((T, d), float("nan"), dtype=h_dt, device="cuda"), torch.full((T, d), float("nan"), dtype=w_dt, device="cuda")
        B.residual_norm(norm, cu(h), cu(y), ho, xo, gate=cu(gate))
        torch.cuda.synchronize()
        o = lambda t: None if t is None else f64(t)  # noqa: E731
        H, X, bh, bx = bounds(f64(h), f64(y), f64(w_pre), o(w_post), o(gate), 0.5, d, h_dt, w_dt)
        within(ho, H, bh, "h")
        within(xo, X, bx, "x")


@pytest.mark.parametrize("T,d,dt", [(257, 4104, BF), (260, 8192, F32), (256, 8184, BF), (300, 512, BF), (70, 1016, F32), (9, 24, BF)])
def test_residual_norm_many_rows(T, d, dt):
    say(f"[norm] T={T} d={d} {dt}")
    g = torch.Generator().manual_seed(d * 7 + T)
    rnd = lambda s, std=1.0: (torch.randn(s, generator=g) * std).to(dt)  # noqa: E731
    h, y, w_pre, w_post, gate = rnd((T, d), 2.0), rnd((T, d)), 1 + rnd((d,), 0.2), 1 + rnd((d,), 0.2), rnd((T, d))
    ho, xo = (torch.full((T, d), float("nan"), dtype=dt, device="cuda") for _ in range(2))
    B.residual_norm(B.ResidualNorm(w_pre.cuda(), w_post=w_post.cuda(), eps=1e-5, scale=0.5), h.cuda(), y.cuda(), ho, xo, gate=gate.cuda())
    torch.cuda.synchronize()
    H, X, bh, bx = bounds(f64(h), f64(y), f64(w_pre), f64(w_post), f64(gate), 0.5, d, dt, dt)
    within(ho, H, bh, "h")
    within(xo, X, bx, "x")


def test_parts_of_it_and_in_place():
    T, d = 9, 1000
    g = torch.Generator().manual_seed(3)
    h, y = torch.randn((T, d), generator=g).cuda(), torch.randn((T, d), generator=g).cuda()
    w = (1 + 0.1 * torch.randn((d,), generator=g)).cuda()
    norm = B.ResidualNorm(w, scale=0.25)
    ho, xo, x_only, h_only = (torch.empty_like(h) for _ in range(4))
    B.residual_norm(norm, h, y, ho, xo)
    B.residual_norm(norm, h, y, None, x_only)  # the norm without the residual
    B.residual_norm(norm, h, y, h_only, None)  # the residual without the norm
    torch.cuda.synchronize()
    assert torch.equal(xo, x_only) and torch.equal(ho, h_only)
    first = torch.empty_like(h)
    B.residual_norm(norm, h, None, None, first)  # no block before it: the norm of h
    torch.cuda.synchronize()
    H, X, _, bx = bounds(f64(h), None, f64(w), None, None, 0.25, d, F32, F32)
    within(first, X, bx, "norm alone")
    h2 = h.clone()
    B.residual_norm(norm, h2, y, h2, xo)
    torch.cuda.synchronize()
    assert torch.equal(h2, ho)
    B.residual_norm(norm, h[:0], y[:0], ho[:0], xo[:0])


def test_rows_of_zeros_and_rows_apart():
    """A row of zeros gives zeros (eps keeps the root from zero); rows do not touch each other,
    whatever is in them."""
    T, d = 4, 4096
    g = torch.Generator().manual_seed(4)
    h, y = torch.randn((T, d), generator=g).to(BF).cuda(), torch.randn((T, d), generator=g).cuda()
    norm = B.ResidualNorm(torch.ones(d, dtype=BF, device="cuda"), w_post=torch.ones(d, dtype=BF, device="cuda"))
    clean_h, clean_x, ho, xo = (torch.empty((T, d), dtype=BF, device="cuda") for _ in range(4))
    B.residual_norm(norm, h, y, clean_h, clean_x)
    h[1], y[1], h[2, 7], y[3, 9] = 0, 0, float("inf"), float("nan")
    B.residual_norm(norm, h, y, ho, xo)
    torch.cuda.synchronize()
    assert torch.equal(ho[0], clean_h[0]) and torch.equal(xo[0], clean_x[0])
    assert (ho[1] == 0).all() and (xo[1] == 0).all()
    assert torch.isnan(xo[3]).all() and torch.isnan(ho[3]).all()
    assert torch.isinf(ho[2, 7]) and torch.isnan(xo[2, 7]) and (xo[2, :7] == 0).all()
