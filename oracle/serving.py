"""What stands between two sparse FFN steps of a decoder layer: the paged key/value cache
(page plan, rotary append, attention) and the residual norm, in numpy float64.

These are the definitions in ``include/sparse_ffn.h``; no source page states them. The
attention function also returns what a rounding-error bound needs.
"""

import numpy as np


def cache_plan(page, table, free_pages, n_free, held, ctx, new, n_pages, max_tokens):
    """One step's plan. ``table`` is a list of lists (each request's held pages in order);
    returns a dict with the new table rows (as lists of the needed pages), the stack, its
    count, cu, kv_len, pos and slot, or ``status`` alone when it cannot be done."""
    up = lambda n: -(-n // page)  # noqa: E731
    cap = len(table[0]) if table else 0
    for h, c, n in zip(held, ctx, new):
        if h < 0 or c < 0 or n < 0 or c > h or h > cap * page or c + n > cap * page:
            return {"status": -1}
    if sum(new) > max_tokens or not 0 <= n_free <= n_pages:
        return {"status": -1}
    stack = list(free_pages[:n_free])
    rows = [list(r) for r in table]
    for r, (h, c, n) in enumerate(zip(held, ctx, new)):
        stack += rows[r][up(c + n):up(h)]
    if len(stack) > n_pages:
        return {"status": -1}
    wanted = sum(max(0, up(c + n) - up(h)) for h, c, n in zip(held, ctx, new))
    if wanted > len(stack):
        return {"status": wanted - len(stack)}
    for r, (h, c, n) in enumerate(zip(held, ctx, new)):
        for e in range(up(h), up(c + n)):
            rows[r][e] = stack.pop()
    cu, pos, slot = [0], [], []
    for r, (c, n) in enumerate(zip(ctx, new)):
        cu.append(cu[-1] + n)
        for p in range(c, c + n):
            pos.append(p)
            slot.append(rows[r][p // page] * page + p % page)
    return {"status": 0, "table": rows, "used": [up(c + n) for c, n in zip(ctx, new)], "stack": stack, "cu": cu,
            "kv_len": [c + n for c, n in zip(ctx, new)], "pos": pos, "slot": slot}


def rotate(x, pos, rope, rot):
    """x [T, heads, dh], rope [n_pos, rot] (cosines, then sines): the first rot values of
    each head turned, value i with value i + rot / 2."""
    x = np.array(x, dtype=np.float64)
    if rot:
        cs = np.asarray(rope, dtype=np.float64)[np.clip(pos, 0, len(rope) - 1)]
        c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
        a, b = x[..., :rot // 2].copy(), x[..., rot // 2:rot].copy()
        x[..., :rot // 2] = a * c - b * s
        x[..., rot // 2:rot] = b * c + a * s
    return x


def attend(q, k, v, n_seen_lo, n_seen_hi, scale):
    """One request: q [n, h_q, dh], k and v [len, h_kv, dh]; token i sees the keys
    n_seen_lo[i] <= j < n_seen_hi[i]. Returns (out, spread, reach): the outputs, and for the
    error bound sum_j w_j |v_j| and the largest 2-norm of the products q_e k_je and largest
    |score| a row meets. A row that sees no key gives zeros."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    n, h_q, dh = q.shape
    g = h_q // k.shape[1]
    out, spread, reach = np.zeros((n, h_q, dh)), np.zeros((n, h_q, dh)), np.zeros((n, h_q, 2))
    for i in range(n):
        lo, hi = max(0, int(n_seen_lo[i])), min(int(n_seen_hi[i]), len(k))
        if hi <= lo:
            continue
        for h in range(h_q):
            kk, vv = k[lo:hi, h // g], v[lo:hi, h // g]
            s = (kk @ q[i, h]) * scale
            w = np.exp(s - s.max())
            w /= w.sum()
            out[i, h] = w @ vv
            spread[i, h] = w @ np.abs(vv)
            reach[i, h, 0] = scale * np.sqrt(((kk * kk) @ (q[i, h] * q[i, h])).max())
            reach[i, h, 1] = np.abs(s).max()
    return out, spread, reach


def seen(kv_len, n, window):
    """First and one-past-last key of each of the n new tokens of a request of kv_len."""
    pos = kv_len - n + np.arange(n)
    return (np.maximum(0, pos - window + 1) if window else np.zeros(n, dtype=int)), np.minimum(pos + 1, kv_len)


def rms_norm(x, w, eps):
    x = np.asarray(x, dtype=np.float64)
    return x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * np.asarray(w, dtype=np.float64)


def residual_norm(h, y, w_pre=None, w_post=None, gate=None, scale=1.0, eps=1e-5):
    """(h_out, x_out): h + scale gate N(y; w_post), and its norm by w_pre."""
    h = np.asarray(h, dtype=np.float64)
    if y is not None:
        u = rms_norm(y, w_post, eps) if w_post is not None else np.asarray(y, dtype=np.float64)
        if gate is not None:
            u = u * np.asarray(gate, dtype=np.float64)
        h = h + scale * u
    return h, None if w_pre is None else rms_norm(h, w_pre, eps)


# ---- the cache in 8 bits --------------------------------------------------------------

EXP_LEAST, EXP_MOST = 10, 246  # a row's byte b stands for 2^(b - 127)


def e4m3_values():
    """What the 256 codes stand for: a sign, 4 bits of exponent (bias 7; 0 for subnormal), 3 of
    significand; 0x7f and 0xff are NaN and there is no infinity."""
    c = np.arange(128)
    v = np.where(c >= 8, (8 + c % 8) * 2.0 ** (c // 8 - 10), (c % 8) * 2.0 ** -9)
    v[127] = np.nan
    return np.concatenate([v, -v])


def stand_for(codes, b):
    """Values of codes [..., dh] and their rows' bytes b [...]."""
    b = np.clip(np.asarray(b, dtype=np.int64), EXP_LEAST, EXP_MOST)
    return e4m3_values()[np.asarray(codes)] * (2.0 ** (b - 127.0))[..., None]


def quantise(x):
    """(codes, bytes) of rows x [..., dh]: per row the least power of two with which 448 times it
    is not below the largest finite magnitude, and of each value the nearest code, ties to the
    even one; magnitudes past the largest code become it, infinities and NaN become NaN."""
    x = np.asarray(x, dtype=np.float64)
    ok = np.isfinite(x)
    top = np.where(ok, np.abs(x), 0.0).max(axis=-1)
    b = np.full(top.shape, EXP_LEAST, dtype=np.int64)
    for e in range(EXP_LEAST, EXP_MOST):
        b = np.where(top > 448.0 * 2.0 ** (e - 127), e + 1, b)
    vals = e4m3_values()[:127]
    y = np.minimum(np.abs(np.where(ok, x, 0.0)) * (2.0 ** (127.0 - b))[..., None], 448.0)
    up = np.minimum(np.searchsorted(vals, y), 126)
    down = np.maximum(up - 1, 0)
    mid = (vals[up] + vals[down]) / 2
    code = np.where((y > mid) | ((y == mid) & (up % 2 == 0)), up, down)
    code = np.where(y == vals[up], up, code)
    return np.where(ok, code + 128 * np.signbit(np.where(ok, x, 0.0)), 127).astype(np.uint8), b.astype(np.uint8)
