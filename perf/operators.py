"""The cases of the serving operators around the sparse FFN step: the paged key/value cache
(its page plan, appends and attention) and the residual norm. Each is computed in its plain
form with elementary torch operations, or, where ``own`` is true, by the library.

plan    page tables, slot maps and positions of one step from the requests' lengths
append  rotary positions of q and k, and the new keys and values written into the cache
attend  attention of each request's new tokens over its cached keys and values
norm    residual update h + scale gate N(y) and the next block's norm of it

Sequence lengths are a function of the case; the seed makes the values, the pages' places
and the stack of free pages.
"""

import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # one decode step of four requests
        {"name": "plan_decode_r4", "op": "plan", "R": 4, "page": 16, "ctx": 2048, "new": 1, "drop": 0},
        # a verification step that drops rejected tokens, and prompts among it: a large server batch
        {"name": "plan_mixed_r1024", "op": "plan", "R": 1024, "page": 16, "ctx": 8192, "new": 48, "drop": 15},
        # the four tokens of a batched decode step (d 4096)
        {"name": "append_t4", "op": "append", "T": 4, "h_q": 32, "h_kv": 8, "dh": 128, "page": 16, "rot": 128, "dtype": "bf16"},
        # prompt tokens of several requests at once (d 8192)
        {"name": "append_t8000", "op": "append", "T": 8000, "h_q": 64, "h_kv": 8, "dh": 128, "page": 64, "rot": 128, "dtype": "bf16"},
        # one request's decode step with a short context, a key head for every query head (d 4096)
        {"name": "attend_r1_short", "op": "attend", "R": 1, "h_q": 32, "h_kv": 32, "dh": 128, "page": 16, "ctx": 500, "new": 1, "ragged": False, "window": 0, "dtype": "bf16"},
        # a serving batch of single tokens with ragged contexts (d 4096)
        {"name": "attend_r48_ragged", "op": "attend", "R": 48, "h_q": 32, "h_kv": 8, "dh": 128, "page": 32, "ctx": 8000, "new": 1, "ragged": True, "window": 0, "dtype": "bf16"},
        # one token over a long context (d 8192)
        {"name": "attend_r1_long", "op": "attend", "R": 1, "h_q": 64, "h_kv": 8, "dh": 128, "page": 64, "ctx": 131000, "new": 1, "ragged": False, "window": 0, "dtype": "bf16"},
        # the 16-token verification chunk of four requests (d 8192)
        {"name": "attend_verify16", "op": "attend", "R": 4, "h_q": 64, "h_kv": 8, "dh": 128, "page": 64, "ctx": 6000, "new": 16, "ragged": True, "window": 0, "dtype": "bf16"},
        # a chunk of a prompt after an earlier part of it (d 4096)
        {"name": "attend_prompt2048", "op": "attend", "R": 2, "h_q": 32, "h_kv": 8, "dh": 128, "page": 64, "ctx": 8192, "new": 2048, "ragged": False, "window": 0, "dtype": "bf16"},
        # a small fp32 model's chunk (d 256) under a sliding window, at odd lengths
        {"name": "attend_f32_window", "op": "attend", "R": 6, "h_q": 4, "h_kv": 2, "dh": 64, "page": 16, "ctx": 1500, "new": 37, "ragged": True, "window": 700, "dtype": "f32"},
        # one token between two blocks (d 4096): the FFN's fp32 output, a bf16 model
        {"name": "norm_t1", "op": "norm", "T": 1, "d": 4096, "h": "f32", "y": "f32", "w": "bf16", "post": False, "gate": 0},
        # prompt tokens (d 8192) with a norm after the block and a gate vector
        {"name": "norm_t8192_gated", "op": "norm", "T": 8192, "d": 8192, "h": "bf16", "y": "f32", "w": "bf16", "post": True, "gate": 1},
    ]


HEADS = [(32, 32), (32, 8), (64, 8), (28, 4), (16, 16), (12, 4), (8, 1), (4, 2)]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend", "attend", "norm"])
    if op == "plan":
        R = _log(rng, 1, 1024)
        return {"op": op, "R": R, "page": rng.choice([16, 32, 64, 128, 256]), "ctx": _log(rng, 40, 8192),
                "new": rng.choice([1, _log(rng, 1, 48)]), "drop": rng.choice([0, rng.randint(1, 15)])}
    if op == "append":
        h_q, h_kv = rng.choice(HEADS)
        dh = 128 if h_q + 2 * h_kv == 48 else rng.choice([64, 128])
        T = _log(rng, 1, min(8000, 8000 * 80 * 128 // ((h_q + 2 * h_kv) * dh * 2)))
        return {"op": op, "T": T, "h_q": h_q, "h_kv": h_kv, "dh": dh, "page": rng.choice([16, 32, 64, 128, 256]),
                "rot": rng.choice([dh, dh, dh // 2]), "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op == "norm":
        d = 8 * _log(rng, 32, 1024)
        d += 8 if d == 3072 else 0
        return {"op": op, "T": _log(rng, 1, 4000), "d": d, "h": rng.choice(["bf16", "f32"]), "y": rng.choice(["bf16", "f32"]),
                "w": rng.choice(["bf16", "bf16", "f32"]), "post": rng.random() < 0.5, "gate": rng.choice([0, 1, 2])}
    h_q, h_kv = rng.choice(HEADS)
    dh = rng.choice([64, 128, 128])
    case = {"op": op, "R": 1, "h_q": h_q, "h_kv": h_kv, "dh": dh, "page": rng.choice([16, 32, 64, 128, 256]), "ctx": 0, "new": 1,
            "ragged": rng.random() < 0.7, "window": rng.choice([0, 0, 0, _log(rng, 100, 4096)]),
            "dtype": rng.choice(["bf16", "bf16", "bf16", "f32"])}
    kind = rng.choice(["decode", "decode", "verify", "prompt"])
    if kind == "prompt":
        case["R"] = _log(rng, 1, 4)
        case["new"] = _log(rng, 17, 2000) // case["R"] + 1
        case["ctx"] = rng.choice([0, _log(rng, 1, 4000)])
    else:
        case["new"] = 1 if kind == "decode" else rng.randint(2, 16)
        case["R"] = _log(rng, 1, 48)
        case["ctx"] = _log(rng, 1, min(100000, 130000 * 1024 // (case["R"] * h_kv * dh * (2 if case["dtype"] == "f32" else 1))))
    return case


# ---- lengths: a function of the case alone ------------------------------------------


def _rng_of(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _attend_lens(case):
    """(tokens before the step, new tokens) of each request."""
    r = _rng_of(case)
    if not case["ragged"]:
        return [case["ctx"]] * case["R"], [case["new"]] * case["R"]
    ctx = [r.randint(0, case["ctx"]) if i else case["ctx"] for i in range(case["R"])]
    new = [r.randint(1, case["new"]) if i else case["new"] for i in range(case["R"])]
    return ctx, new


def _plan_lens(case):
    """(tokens the pages were taken for, tokens kept of them, new tokens) of each request; one in sixteen is new."""
    r = _rng_of(case)
    held = [0 if i % 16 == 15 else _log(r, 1, case["ctx"]) for i in range(case["R"])]
    kept = [max(0, h - r.randint(0, case["drop"])) for h in held]
    new = [r.randint(1, case["new"]) for _ in held]
    return held, kept, new


def _ceil(a, b):
    return -(-a // b)


def _pairs(lo, n):
    """Keys seen by n tokens that see lo + 1, lo + 2, ... of them."""
    return n * lo + n * (n + 1) // 2


# ---- inputs -------------------------------------------------------------------------


def _randn(g, shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = globals()["_prepare_" + case["op"]](case, g)
    s["case"] = case
    if own:  # the handles that a user's program makes once
        from contextual_activation_sparsity_amd import binding

        s["B"] = binding
        if case["op"] == "norm":
            s["norm"] = binding.ResidualNorm(s["w_pre"], w_post=s["w_post"], eps=EPS, scale=s["scale"])
        else:
            s["cache"] = binding.KVCache(s["k_cache"], s["v_cache"])
        if case["op"] == "attend":
            nbytes = binding.kv_cache_attend_workspace_size(s["cache"], case["R"], s["q"].shape[0], case["h_q"], s["max_new"], s["max_len"])
            s["ws"] = binding.workspace(nbytes)
    return s


def _prepare_plan(case, g):
    held, kept, new = _plan_lens(case)
    R, p = case["R"], case["page"]
    pages = [_ceil(h, p) for h in held]
    need = [_ceil(c + n, p) for c, n in zip(kept, new)]
    max_pages = max(max(pages), max(need))
    n_pages = sum(pages) + sum(max(0, m - h) for m, h in zip(need, pages)) + 64
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor([0] + pages, device="cuda").cumsum(0)[:-1]
    at = torch.arange(max_pages, device="cuda")
    mine = at[None, :] < torch.tensor(pages, device="cuda")[:, None]
    table = torch.where(mine, order[(first[:, None] + at[None, :]).clamp(max=n_pages - 1)], torch.full((), -1, dtype=torch.int32, device="cuda"))
    n_free = n_pages - sum(pages)
    free = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
    free[:n_free] = order[sum(pages):]
    T = sum(new)
    # the cache itself: a plan only needs its shape, so one short head stands for it
    k_cache = torch.zeros((n_pages, 1, p, 64), dtype=torch.bfloat16, device="cuda")
    out = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"k_cache": k_cache, "v_cache": torch.zeros_like(k_cache), "held": _i32(held), "kept": _i32(kept), "new": _i32(new),
            "table": table.contiguous(), "free": free, "n_free": _i32([n_free]), "n_free_out": out(1), "cu": out(R + 1),
            "kv_len": out(R), "pos": out(T), "slot": out(T), "status": out(1)}


def _prepare_append(case, g):
    T, h_q, h_kv, dh, p = case["T"], case["h_q"], case["h_kv"], case["dh"], case["page"]
    dt = DTYPES[case["dtype"]]
    used = _ceil(T, p)
    n_pages = used + used // 4 + 2
    qkv = _randn(g, (T, h_q + 2 * h_kv, dh), dt)  # the fused projection's output
    k_cache, v_cache = _randn(g, (n_pages, h_kv, p, dh), dt), _randn(g, (n_pages, h_kv, p, dh), dt)
    pages = torch.randperm(n_pages, generator=g, device="cuda")
    i = torch.arange(T, device="cuda")
    slot = (pages[i // p] * p + i % p).to(torch.int32)
    n_pos = 8192
    pos = ((i + int(torch.randint(0, n_pos, (1,), generator=g, device="cuda"))) % n_pos).to(torch.int32)
    inv = 10000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"])
    ang = torch.arange(n_pos, device="cuda", dtype=torch.float64)[:, None] * inv[None, :]
    rope = torch.cat([ang.cos(), ang.sin()], 1).to(torch.float32).contiguous()
    return {"k_cache": k_cache, "v_cache": v_cache, "q": qkv[:, :h_q], "k": qkv[:, h_q:h_q + h_kv], "v": qkv[:, h_q + h_kv:],
            "pos": pos, "slot": slot, "rope": rope, "q_out": torch.empty((T, h_q, dh), dtype=dt, device="cuda")}


def _prepare_attend(case, g):
    ctx, new = _attend_lens(case)
    R, h_q, h_kv, dh, p = case["R"], case["h_q"], case["h_kv"], case["dh"], case["page"]
    dt = DTYPES[case["dtype"]]
    lens = [c + n for c, n in zip(ctx, new)]
    pages = [_ceil(n, p) for n in lens]
    max_pages = max(pages)
    n_pages = sum(pages) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor([0] + pages, device="cuda").cumsum(0)[:-1]
    at = torch.arange(max_pages, device="cuda")
    mine = at[None, :] < torch.tensor(pages, device="cuda")[:, None]
    table = torch.where(mine, order[(first[:, None] + at[None, :]).clamp(max=n_pages - 1)], torch.full((), -1, dtype=torch.int32, device="cuda"))
    # keys around a mean of their own for each head, as trained models have them; queries sharp enough that the weights differ
    k_cache = _randn(g, (n_pages, h_kv, p, dh), dt)
    k_cache += _randn(g, (1, h_kv, 1, dh), dt)
    v_cache = _randn(g, (n_pages, h_kv, p, dh), dt)
    T = sum(new)
    q = _randn(g, (T, h_q, dh), dt, std=2.0)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return {"k_cache": k_cache, "v_cache": v_cache, "q": q, "table": table.contiguous(), "cu": _i32(cu), "kv_len": _i32(lens),
            "max_new": max(new), "max_len": max(lens), "out": torch.empty((T, h_q, dh), dtype=dt, device="cuda")}


def _prepare_norm(case, g):
    T, d, w = case["T"], case["d"], DTYPES[case["w"]]
    gate = None if not case["gate"] else _randn(g, (d,) if case["gate"] == 1 else (T, d), w)
    return {"h": _randn(g, (T, d), DTYPES[case["h"]], 2.0), "y": _randn(g, (T, d), DTYPES[case["y"]], 0.7),
            "w_pre": 1 + _randn(g, (d,), w, 0.1), "w_post": 1 + _randn(g, (d,), w, 0.1) if case["post"] else None, "gate": gate,
            "scale": 0.5 if case["post"] else 1.0, "h_out": torch.empty((T, d), dtype=DTYPES[case["h"]], device="cuda"),
            "x_out": torch.empty((T, d), dtype=w, device="cuda")}


# ---- one pass -----------------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    if not own:
        return globals()["_plain_" + op](state)
    B, s = state["B"], state
    if op == "plan":
        B.kv_cache_plan(s["cache"], s["held"], s["kept"], s["new"], s["table"], s["free"], s["n_free"], s["n_free_out"], s["cu"], s["kv_len"],
                        s["pos"], s["slot"], s["status"])
        return {k: s[k] for k in ("table", "free", "n_free_out", "cu", "kv_len", "pos", "slot", "status")}
    if op == "append":
        B.kv_cache_append(s["cache"], s["k"], s["v"], s["slot"], q=s["q"], q_out=s["q_out"], pos=s["pos"], rope=s["rope"])
        return {k: s[k] for k in ("q_out", "k_cache", "v_cache")}
    if op == "attend":
        B.kv_cache_attend(s["cache"], s["q"], s["table"], s["cu"], s["kv_len"], s["out"], s["ws"], s["max_new"], s["max_len"],
                          window=s["case"]["window"])
        return s["out"]
    B.residual_norm(s["norm"], s["h"], s["y"], s["h_out"], s["x_out"], gate=s["gate"])
    return {k: s[k] for k in ("h_out", "x_out")}


def _plain_plan(s):
    p, table, free = s["case"]["page"], s["table"], s["free"]
    held, kept, new = s["held"].long(), s["kept"].long(), s["new"].long()
    have, need = (held + p - 1) // p, (kept + new + p - 1) // p
    rel, take = (have - need).clamp(min=0), (need - have).clamp(min=0)
    rel_end, take_end = rel.cumsum(0), take.cumsum(0)
    # the pages given back, in order: number i of them is entry need + (i - those before) of its request
    i = torch.arange(free.shape[0], device=free.device)
    r = torch.searchsorted(rel_end, i, right=True).clamp(max=held.shape[0] - 1)
    at = (need[r] + i - (rel_end - rel)[r]).clamp(0, table.shape[1] - 1)
    back = table[r, at]
    n = s["n_free"].long()
    # pushed on the stack, then popped: number j of the taken pages is entry n + given - 1 - j
    j = (take_end - take)[:, None] + torch.arange(table.shape[1], device=free.device)[None, :] - have[:, None]
    top = n + rel_end[-1:] - 1 - j
    page = torch.where(top >= n, back[(top - n).clamp(0, free.shape[0] - 1)], free[top.clamp(0, free.shape[0] - 1)])
    e = torch.arange(table.shape[1], device=free.device)[None, :]
    table = torch.where((e >= have[:, None]) & (e < need[:, None]), page, table)
    n_out = n + rel_end[-1:] - take_end[-1:]
    free = torch.where((i >= n) & (i < n_out), back[(i - n).clamp(min=0)], free)
    end = new.cumsum(0)
    t = torch.arange(s["pos"].shape[0], device=free.device)
    q = torch.searchsorted(end, t, right=True)
    pos = kept[q] + t - (end - new)[q]
    slot = table[q, pos // p].long() * p + pos % p
    cu = torch.cat([torch.zeros_like(end[:1]), end])
    to = lambda x: x.to(torch.int32)  # noqa: E731
    return {"table": table, "free": free, "n_free_out": to(n_out), "cu": to(cu), "kv_len": to(kept + new), "pos": to(pos), "slot": to(slot),
            "status": torch.zeros_like(s["status"])}


def _plain_rope(x, cs, rot):
    x = x.float()
    c, n = cs[:, None, : rot // 2], cs[:, None, rot // 2:]
    a, b = x[..., : rot // 2], x[..., rot // 2: rot]
    return torch.cat([a * c - b * n, b * c + a * n, x[..., rot:]], -1)


def _plain_append(s):
    rot, p = s["case"]["rot"], s["case"]["page"]
    cs = s["rope"][s["pos"].long()]
    slot = s["slot"].long()
    s["k_cache"][slot // p, :, slot % p] = _plain_rope(s["k"], cs, rot).to(s["k"].dtype)
    s["v_cache"][slot // p, :, slot % p] = s["v"]
    return {"q_out": _plain_rope(s["q"], cs, rot).to(s["q"].dtype), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attend(s):
    """Every request padded to the longest: its pages gathered, the scores of all its tokens, a mask, the weights, their sum of the values."""
    q, table, R, n, L, window = s["q"], s["table"].long(), s["case"]["R"], s["max_new"], s["max_len"], s["case"]["window"]
    T, h_q, dh = q.shape
    h_kv = s["k_cache"].shape[1]
    g = h_q // h_kv
    k = s["k_cache"][table].transpose(1, 2).reshape(R, h_kv, -1, dh)[:, :, :L].float()
    v = s["v_cache"][table].transpose(1, 2).reshape(R, h_kv, -1, dh)[:, :, :L].float()
    cu, lens = s["cu"].long(), s["kv_len"].long()
    i = torch.arange(n, device=q.device)
    rows = (cu[:-1, None] + i[None, :]).clamp(max=T - 1)  # [R, n]
    qp = q[rows].float().reshape(R, n, h_kv, g, dh).permute(0, 2, 3, 1, 4).reshape(R, h_kv, g * n, dh)
    scores = torch.matmul(qp, k.transpose(2, 3)) * (dh ** -0.5)
    pos = (lens - (cu[1:] - cu[:-1]))[:, None] + i[None, :]  # [R, n]
    j = torch.arange(L, device=q.device)
    seen = (j[None, None, :] <= pos[:, :, None]) & (j[None, None, :] < lens[:, None, None])
    if window:
        seen &= j[None, None, :] > pos[:, :, None] - window
    scores = scores.reshape(R, h_kv, g, n, L).masked_fill(~seen[:, None, None], float("-inf"))
    w = (scores - scores.amax(-1, keepdim=True).clamp(min=-1e30)).exp()
    w = w / w.sum(-1, keepdim=True).clamp(min=1e-30)
    o = torch.matmul(w.reshape(R, h_kv, g * n, L), v).reshape(R, h_kv, g, n, dh).permute(0, 3, 1, 2, 4).reshape(R, n, h_q, dh)
    t = torch.arange(T, device=q.device)
    r = torch.searchsorted(cu[1:], t, right=True)
    return o[r, t - cu[r]].to(q.dtype)


def _plain_norm(s):
    y = s["y"].float()
    if s["w_post"] is not None:
        y = y * (y.square().mean(-1, keepdim=True) + EPS).rsqrt() * s["w_post"].float()
    if s["gate"] is not None:
        y = y * s["gate"].float()
    h = s["h"].float() + s["scale"] * y
    x = h * (h.square().mean(-1, keepdim=True) + EPS).rsqrt() * s["w_pre"].float()
    return {"h_out": h.to(s["h"].dtype), "x_out": x.to(s["w_pre"].dtype)}


# ---- what a pass cannot do without --------------------------------------------------


def _size(name):
    return 2 if name == "bf16" else 4


def work(case):
    op = case["op"]
    if op == "plan":
        held, kept, new = _plan_lens(case)
        p, T = case["page"], sum(new)
        pages = [(_ceil(h, p), _ceil(c + n, p)) for h, c, n in zip(held, kept, new)]
        read = sum(_ceil(c + n, p) - c // p for c, n in zip(kept, new)) + sum(max(0, h - m) for h, m in pages)
        moved = sum(abs(m - h) for h, m in pages)
        return {"bytes": 12 * case["R"] + 4 * read + 8 * T + 8 * case["R"] + 4 * moved, "flops": 0}
    if op == "append":
        n, e = case["T"] * (case["h_q"] + 2 * case["h_kv"]) * case["dh"], _size(case["dtype"])
        return {"bytes": 2 * n * e + case["T"] * (4 * case["rot"] + 8), "flops": 3 * case["T"] * (case["h_q"] + case["h_kv"]) * case["rot"]}
    if op == "norm":
        n, w = case["T"] * case["d"], _size(case["w"])
        vec = case["d"] * w * (1 + case["post"] + (case["gate"] == 1))
        return {"bytes": n * (2 * _size(case["h"]) + _size(case["y"]) + w + (w if case["gate"] == 2 else 0)) + vec, "flops": 10 * n}
    ctx, new = _attend_lens(case)
    e, W = _size(case["dtype"]), case["window"]
    keys = pairs = 0
    for c, n in zip(ctx, new):
        first = max(0, c + 1 - W) if W else 0
        keys += c + n - first
        full = min(n, max(0, W - c)) if W else n  # tokens that see everything before them
        pairs += _pairs(c, full) + (n - full) * W
    T = sum(new)
    return {"bytes": e * case["dh"] * (2 * keys * case["h_kv"] + 2 * T * case["h_q"]), "flops": 4 * pairs * case["h_q"] * case["dh"]}


# ---- the definitions, in 64 bits ----------------------------------------------------


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = globals()["_prepare_" + case["op"]](case, g)
    return globals()["_exact_" + case["op"]](case, s)


def _exact_append(case, s):
    rot, p = case["rot"], case["page"]
    at = s["pos"].long()
    m = torch.complex(s["rope"][at, : rot // 2].double(), s["rope"][at, rot // 2:].double())[:, None, :]

    def turn(x):
        x = x.double()
        z = torch.complex(x[..., : rot // 2].contiguous(), x[..., rot // 2: rot].contiguous()) * m
        return torch.cat([z.real, z.imag, x[..., rot:]], -1)

    k, v, slot = s["k_cache"].double(), s["v_cache"].double(), s["slot"].long()
    flat = lambda c: c.permute(0, 2, 1, 3).reshape(-1, case["h_kv"], case["dh"])  # noqa: E731
    back = lambda c: c.reshape(-1, p, case["h_kv"], case["dh"]).permute(0, 2, 1, 3).contiguous()  # noqa: E731
    k, v = flat(k).index_copy(0, slot, turn(s["k"])), flat(v).index_copy(0, slot, s["v"].double())
    return {"q_out": turn(s["q"]), "k_cache": back(k), "v_cache": back(v)}


def _exact_attend(case, s):
    h_kv, g, dh, p, W = case["h_kv"], case["h_q"] // case["h_kv"], case["dh"], case["page"], case["window"]
    ctx, new = _attend_lens(case)
    out, t0 = [], 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        pages = s["table"][r, : _ceil(c + n, p)].long()
        k = s["k_cache"][pages].double().permute(1, 0, 2, 3).reshape(h_kv, -1, dh)[:, : c + n]
        v = s["v_cache"][pages].double().permute(1, 0, 2, 3).reshape(h_kv, -1, dh)[:, : c + n]
        q = s["q"][t0:t0 + n].double().reshape(n, h_kv, g, dh)
        t0 += n
        a = torch.arange(c + n, device=k.device)
        heads = []
        for h in range(h_kv):
            x = (q[:, h].reshape(n * g, dh) @ k[h].t()).reshape(n, g, c + n) / dh ** 0.5
            far = a[None, :] - (c + torch.arange(n, device=k.device))[:, None]  # key minus token position
            x = x + torch.where((far > 0) | ((far <= -W) if W else (far > 0)), float("-inf"), 0.0)[:, None, :]
            heads.append((torch.softmax(x, -1).reshape(n * g, c + n) @ v[h]).reshape(n, g, dh))
        out.append(torch.stack(heads, 1).reshape(n, case["h_q"], dh))
    return torch.cat(out)


def _exact_norm(case, s):
    y = s["y"].double()
    if case["post"]:
        y = s["w_post"].double() * y / torch.sqrt((y * y).sum(1, keepdim=True) / case["d"] + EPS)
    h = s["h"].double() + s["scale"] * (y if s["gate"] is None else y * s["gate"].double())
    return {"h_out": h, "x_out": s["w_pre"].double() * h / torch.sqrt((h * h).sum(1, keepdim=True) / case["d"] + EPS)}
