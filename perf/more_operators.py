"""The cases of the paged cache in 8 bits and of attention over a shared prefix. Each is computed
in its plain form with elementary torch operations, or, where ``own`` is true, by the library.

append8  rotary positions of q and k; the new keys and values written into the cache as e4m3
         values, each head's row of a token with one power of two of its own
read8    tokens' keys and values out of that cache again, by slots
attend8  attention of each request's new tokens over their keys and values in that cache
shared   attention of requests whose first tokens are the same (a system prompt, a document),
         which are read once for all of them; over a cache in the model's type or in 8 bits

A row's power of two is held as one byte b for 2^(b - 127): the smallest one with which the row's
largest magnitude is at most 448 (the largest e4m3 value), 10 at least and 246 at most.

Sequence lengths are a function of the case; the seed makes the values and the pages' places.
"""

import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
N_POS = 8192  # positions of the rotary table


def listed():
    return [
        # the four tokens of a batched decode step (d 4096)
        {"name": "append8_t4", "op": "append8", "T": 4, "h_q": 32, "h_kv": 8, "dh": 128, "page": 16, "rot": 128, "dtype": "bf16"},
        # prompts of a small fp32 model, half of each head turned
        {"name": "append8_f32_t901", "op": "append8", "T": 901, "h_q": 12, "h_kv": 4, "dh": 64, "page": 32, "rot": 32, "dtype": "f32"},
        # prompt tokens of several requests at once (d 8192)
        {"name": "append8_t8000", "op": "append8", "T": 8000, "h_q": 64, "h_kv": 8, "dh": 128, "page": 64, "rot": 128, "dtype": "bf16"},
        # the 16 tokens of a verified chunk, read back
        {"name": "read8_t16", "op": "read8", "T": 16, "h_kv": 8, "dh": 128, "page": 16, "dtype": "bf16"},
        # a long sequence read back, to be kept elsewhere while its request waits
        {"name": "read8_t60000", "op": "read8", "T": 60000, "h_kv": 8, "dh": 128, "page": 64, "dtype": "bf16"},
        # one request's decode step with a short context, a key head for every query head (d 4096)
        {"name": "attend8_r1_short", "op": "attend8", "R": 1, "h_q": 32, "h_kv": 32, "dh": 128, "page": 16, "ctx": 500, "new": 1, "ragged": False, "window": 0, "dtype": "bf16"},
        # a serving batch of single tokens with ragged contexts (d 4096)
        {"name": "attend8_r48_ragged", "op": "attend8", "R": 48, "h_q": 32, "h_kv": 8, "dh": 128, "page": 32, "ctx": 8000, "new": 1, "ragged": True, "window": 0, "dtype": "bf16"},
        # one token over a long context (d 8192)
        {"name": "attend8_r1_long", "op": "attend8", "R": 1, "h_q": 64, "h_kv": 8, "dh": 128, "page": 64, "ctx": 131000, "new": 1, "ragged": False, "window": 0, "dtype": "bf16"},
        # a chunk of a prompt after an earlier part of it (d 4096)
        {"name": "attend8_prompt2048", "op": "attend8", "R": 2, "h_q": 32, "h_kv": 8, "dh": 128, "page": 64, "ctx": 8192, "new": 2048, "ragged": False, "window": 0, "dtype": "bf16"},
        # a small fp32 model: six requests after a common prompt, chunks of odd lengths
        {"name": "shared_f32_r6", "op": "shared", "R": 6, "h_q": 4, "h_kv": 2, "dh": 64, "page": 16, "prefix": 700, "ctx": 90, "new": 5, "ragged": True, "cache": "own", "dtype": "f32"},
        # a serving batch of single tokens that has a long prompt in common (d 4096)
        {"name": "shared_r48", "op": "shared", "R": 48, "h_q": 32, "h_kv": 8, "dh": 128, "page": 32, "prefix": 8000, "ctx": 1000, "new": 1, "ragged": True, "cache": "own", "dtype": "bf16"},
        # verification chunks of many requests over one long document in the 8-bit cache (d 8192)
        {"name": "shared8_verify16_r32", "op": "shared", "R": 32, "h_q": 64, "h_kv": 8, "dh": 128, "page": 64, "prefix": 60001, "ctx": 700, "new": 16, "ragged": True, "cache": "e4m3", "dtype": "bf16"},
    ]


HEADS = [(32, 32), (32, 8), (64, 8), (28, 4), (16, 16), (12, 4), (8, 1), (4, 2)]
PAGES = [16, 32, 64, 128, 256]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["append8", "read8", "attend8", "attend8", "shared", "shared"])
    h_q, h_kv = rng.choice(HEADS)
    dh, page = rng.choice([64, 128, 128]), rng.choice(PAGES)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "append8":
        T = _log(rng, 1, min(8000, 8000 * 80 * 128 // ((h_q + 2 * h_kv) * dh * 2)))
        return {"op": op, "T": T, "h_q": h_q, "h_kv": h_kv, "dh": dh, "page": page, "rot": rng.choice([dh, dh, dh // 2]), "dtype": dtype}
    if op == "read8":
        return {"op": op, "T": _log(rng, 1, min(60000, 60000 * 8 * 128 // (h_kv * dh * 2))), "h_kv": h_kv, "dh": dh, "page": page, "dtype": dtype}
    case = {"op": op, "R": 1, "h_q": h_q, "h_kv": h_kv, "dh": dh, "page": page}
    kind = rng.choice(["decode", "decode", "verify", "prompt"])
    new = 1 if kind == "decode" else rng.randint(2, 16)
    if op == "attend8":
        case |= {"ctx": 0, "new": new, "ragged": rng.random() < 0.7, "window": rng.choice([0, 0, 0, _log(rng, 100, 4096)]), "dtype": dtype}
        if kind == "prompt":
            case["R"] = _log(rng, 1, 4)
            case["new"] = _log(rng, 17, 2000) // case["R"] + 1
            case["ctx"] = rng.choice([0, _log(rng, 1, 4000)])
        else:
            case["R"] = _log(rng, 1, 48)
            case["ctx"] = _log(rng, 1, min(100000, 130000 * 1024 // (case["R"] * h_kv * dh)))
        return case
    if kind == "prompt":
        case["R"] = _log(rng, 2, 8)
        new = _log(rng, 17, 600) // case["R"] + 1
    else:
        case["R"] = _log(rng, 2, 64 if kind == "decode" else 32)
    case |= {"prefix": _log(rng, 300, 60000), "ctx": _log(rng, 1, 1500), "new": new, "ragged": rng.random() < 0.7,
             "cache": rng.choice(["own", "e4m3"]), "dtype": dtype}
    most = 4 * 512 * 64 * 128 * 60000 // (8 if dtype == "f32" else 1)  # what the largest listed case computes; fp32 products take longer
    case["prefix"] = max(300, min(case["prefix"], most // (4 * case["R"] * new * h_q * dh)))
    return case


# ---- lengths: a function of the case alone ------------------------------------------


def _lens(case):
    """(tokens before the step and after the prefix, new tokens) of each request."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    if not case["ragged"]:
        return [case["ctx"]] * case["R"], [case["new"]] * case["R"]
    ctx = [r.randint(0, case["ctx"]) if i else case["ctx"] for i in range(case["R"])]
    new = [r.randint(1, case["new"]) if i else case["new"] for i in range(case["R"])]
    return ctx, new


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


def _random_cache8(g, shape, mean=None):
    """An 8-bit cache as appends leave it: rows of different sizes around a mean for each head."""
    x = torch.randn(shape, generator=g, device="cuda")
    if mean is not None:
        x += mean
    x *= torch.exp(0.5 * torch.randn(shape[:-1] + (1,), generator=g, device="cuda"))
    b = ((x.abs().amax(-1).view(torch.int32) + 0x1FFFFF) >> 23) - 8
    codes = (x * ((254 - b) << 23).view(torch.float32)[..., None]).to(E4M3)
    return codes, b.to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = globals()["_prepare_" + case["op"]](case, g)
    s["case"] = case
    if own:  # the handles that a user's program makes once
        from contextual_activation_sparsity_amd import binding

        s["B"] = binding
        if "k_exp" in s:
            s["cache"] = binding.KVCache8(s["k_cache"], s["v_cache"], s["k_exp"], s["v_exp"], DTYPES[case["dtype"]])
        else:
            s["cache"] = binding.KVCache(s["k_cache"], s["v_cache"])
        if case["op"] == "attend8":
            nbytes = binding.kv8_cache_attend_workspace_size(s["cache"], case["R"], s["q"].shape[0], case["h_q"], s["max_new"], s["max_len"])
            s["ws"] = binding.workspace(nbytes)
        if case["op"] == "shared":
            size = binding.kv8_cache_attend_shared_workspace_size if "k_exp" in s else binding.kv_cache_attend_shared_workspace_size
            s["ws"] = binding.workspace(size(s["cache"], case["R"], s["q"].shape[0], case["h_q"], s["max_new"], case["prefix"], s["max_own"]))
    return s


def _slots(T, p, g):
    """Places of T tokens on shuffled pages, and the number of pages."""
    used = _ceil(T, p)
    n_pages = used + used // 4 + 2
    pages = torch.randperm(n_pages, generator=g, device="cuda")
    i = torch.arange(T, device="cuda")
    return (pages[i // p] * p + i % p).to(torch.int32), n_pages


def _prepare_append8(case, g):
    T, h_q, h_kv, dh, p = case["T"], case["h_q"], case["h_kv"], case["dh"], case["page"]
    dt = DTYPES[case["dtype"]]
    slot, n_pages = _slots(T, p, g)
    qkv = _randn(g, (T, h_q + 2 * h_kv, dh), dt)  # the fused projection's output
    k_cache, k_exp = _random_cache8(g, (n_pages, h_kv, p, dh))
    v_cache, v_exp = _random_cache8(g, (n_pages, h_kv, p, dh))
    i = torch.arange(T, device="cuda")
    pos = ((i + int(torch.randint(0, N_POS, (1,), generator=g, device="cuda"))) % N_POS).to(torch.int32)
    inv = 10000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"])
    ang = torch.arange(N_POS, device="cuda", dtype=torch.float64)[:, None] * inv[None, :]
    rope = torch.cat([ang.cos(), ang.sin()], 1).to(torch.float32).contiguous()
    return {"k_cache": k_cache, "v_cache": v_cache, "k_exp": k_exp, "v_exp": v_exp, "q": qkv[:, :h_q], "k": qkv[:, h_q:h_q + h_kv],
            "v": qkv[:, h_q + h_kv:], "pos": pos, "slot": slot, "rope": rope, "q_out": torch.empty((T, h_q, dh), dtype=dt, device="cuda")}


def _prepare_read8(case, g):
    T, h_kv, dh, p = case["T"], case["h_kv"], case["dh"], case["page"]
    slot, n_pages = _slots(T, p, g)
    k_cache, k_exp = _random_cache8(g, (n_pages, h_kv, p, dh))
    v_cache, v_exp = _random_cache8(g, (n_pages, h_kv, p, dh))
    rows = torch.empty((T, 2 * h_kv, dh), dtype=DTYPES[case["dtype"]], device="cuda")
    return {"k_cache": k_cache, "v_cache": v_cache, "k_exp": k_exp, "v_exp": v_exp, "slot": slot, "k_out": rows[:, :h_kv], "v_out": rows[:, h_kv:]}


def _table(pages, order):
    """Each request's pages one after the other from `order`, in rows of the longest, the rest -1."""
    first = torch.tensor([0] + pages, device="cuda").cumsum(0)[:-1]
    at = torch.arange(max(pages), device="cuda")
    mine = at[None, :] < torch.tensor(pages, device="cuda")[:, None]
    return torch.where(mine, order[(first[:, None] + at[None, :]).clamp(max=order.shape[0] - 1)], torch.full((), -1, dtype=torch.int32, device="cuda"))


def _fill_cache(case, g, n_pages, e4m3):
    shape = (n_pages, case["h_kv"], case["page"], case["dh"])
    # keys around a mean of their own for each head, as trained models have them
    mean = _randn(g, (1, case["h_kv"], 1, case["dh"]))
    if e4m3:
        k_cache, k_exp = _random_cache8(g, shape, mean)
        v_cache, v_exp = _random_cache8(g, shape)
        return {"k_cache": k_cache, "v_cache": v_cache, "k_exp": k_exp, "v_exp": v_exp}
    dt = DTYPES[case["dtype"]]
    return {"k_cache": (_randn(g, shape) + mean).to(dt), "v_cache": _randn(g, shape, dt)}


def _tokens(case, g, new):
    # queries sharp enough that the weights differ
    T, dt = sum(new), DTYPES[case["dtype"]]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return {"q": _randn(g, (T, case["h_q"], case["dh"]), dt, std=2.0), "cu": _i32(cu), "max_new": max(new),
            "out": torch.empty((T, case["h_q"], case["dh"]), dtype=dt, device="cuda")}


def _prepare_attend8(case, g):
    ctx, new = _lens(case)
    lens = [c + n for c, n in zip(ctx, new)]
    pages = [_ceil(n, case["page"]) for n in lens]
    n_pages = sum(pages) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    s = _fill_cache(case, g, n_pages, True)
    return s | _tokens(case, g, new) | {"table": _table(pages, order).contiguous(), "kv_len": _i32(lens), "max_len": max(lens)}


def _prepare_shared(case, g):
    """The prefix's whole pages are every request's first ones; a last page that it fills in part
    is held once by each request, so its few tokens count as the request's own."""
    ctx, new = _lens(case)
    p, prefix = case["page"], case["prefix"]
    common, over = prefix // p, prefix % p
    own_len = [over + c + n for c, n in zip(ctx, new)]
    pages = [_ceil(n, p) for n in own_len]
    n_pages = common + sum(pages) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.cat([order[:common].expand(case["R"], common), _table(pages, order[common:])], 1).contiguous()
    s = _fill_cache(case, g, n_pages, case["cache"] == "e4m3")
    return s | _tokens(case, g, new) | {"table": table, "prefix": table[0].clone(), "kv_len": _i32([common * p + n for n in own_len]), "max_own": max(own_len),
                                        "shared_len": _i32([common * p])}


# ---- one pass -----------------------------------------------------------------------


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        return globals()["_plain_" + op](s)
    B = s["B"]
    if op == "append8":
        B.kv8_cache_append(s["cache"], s["k"], s["v"], s["slot"], q=s["q"], q_out=s["q_out"], pos=s["pos"], rope=s["rope"])
        return {k: s[k] for k in ("q_out", "k_cache", "v_cache", "k_exp", "v_exp")}
    if op == "read8":
        B.kv8_cache_read(s["cache"], s["slot"], s["k_out"], s["v_out"])
        return {k: s[k] for k in ("k_out", "v_out")}
    if op == "attend8":
        B.kv8_cache_attend(s["cache"], s["q"], s["table"], s["cu"], s["kv_len"], s["out"], s["ws"], s["max_new"], s["max_len"],
                           window=case["window"])
        return s["out"]
    call = B.kv8_cache_attend_shared if "k_exp" in s else B.kv_cache_attend_shared
    call(s["cache"], s["q"], s["prefix"], s["shared_len"], s["table"], s["cu"], s["kv_len"], s["out"], s["ws"], s["max_new"], case["prefix"],
         s["max_own"])
    return s["out"]


def _plain_rope(x, cs, rot):
    c, n = cs[:, None, : rot // 2], cs[:, None, rot // 2:]
    a, b = x[..., : rot // 2], x[..., rot // 2: rot]
    return torch.cat([a * c - b * n, b * c + a * n, x[..., rot:]], -1)


def _quantise(x):
    """Rows of float64 values as e4m3 codes and their bytes b; each value rounded once, to the
    nearest, ties to the even one. In 64 bits, where values stand next to a border."""
    a = x.abs().amax(-1)
    m, e = torch.frexp(a)
    b = torch.where(a > 0, e + 127 - 9 + (m > 0.875).to(e.dtype), 0).clamp(10, 246)
    y = torch.ldexp(x, 127 - b[..., None])
    step = torch.ldexp(torch.ones_like(y), (torch.frexp(y)[1] - 1).clamp(min=-6) - 3)
    return (torch.round(y / step) * step).float().to(E4M3), b.to(torch.uint8)


def _plain_append8(s):
    rot, p = s["case"]["rot"], s["case"]["page"]
    cs = s["rope"][s["pos"].long()]
    slot = s["slot"].long()
    at, off = slot // p, slot % p
    for name, x in (("k", _plain_rope(s["k"].double(), cs.double(), rot)), ("v", s["v"].double())):
        codes, b = _quantise(x)
        s[name + "_cache"].view(torch.uint8)[at, :, off] = codes.view(torch.uint8)
        s[name + "_exp"][at, :, off] = b
    q_out = _plain_rope(s["q"].float(), cs, rot).to(s["q"].dtype)
    return {"q_out": q_out} | {k: s[k] for k in ("k_cache", "v_cache", "k_exp", "v_exp")}


def _values(codes, b):
    """What codes (as bytes) and their rows' bytes b stand for, in 32 bits."""
    return codes.view(E4M3).float() * (b.to(torch.int32) << 23).view(torch.float32)[..., None]


def _plain_read8(s):
    p = s["case"]["page"]
    at, off = s["slot"].long() // p, s["slot"].long() % p
    return {n + "_out": _values(s[n + "_cache"].view(torch.uint8)[at, :, off], s[n + "_exp"][at, :, off]).to(s["k_out"].dtype) for n in ("k", "v")}


def _pages(s, name, pages):
    """Keys or values of the pages, in 32 bits: [..., pages, h_kv, page, dh]."""
    if "k_exp" in s:
        return _values(s[name + "_cache"].view(torch.uint8)[pages], s[name + "_exp"][pages])
    return s[name + "_cache"][pages].float()


def _padded(s):
    """The tokens' queries padded to the longest request, [R, h_kv, g n, dh], and each row of q's place there."""
    q, cu, R, n = s["q"], s["cu"].long(), s["case"]["R"], s["max_new"]
    T, h_q, dh = q.shape
    h_kv = s["case"]["h_kv"]
    g = h_q // h_kv
    i = torch.arange(n, device=q.device)
    rows = (cu[:-1, None] + i[None, :]).clamp(max=T - 1)  # [R, n]
    qp = q[rows].float().reshape(R, n, h_kv, g, dh).permute(0, 2, 3, 1, 4).reshape(R, h_kv, g * n, dh) * dh ** -0.5
    t = torch.arange(T, device=q.device)
    r = torch.searchsorted(cu[1:], t, right=True)
    return qp, r, t - cu[r]


def _plain_attend8(s):
    """Every request padded to the longest: its pages gathered, the scores of all its tokens, a mask, the weights, their sum of the values."""
    case, L, n = s["case"], s["max_len"], s["max_new"]
    R, h_q, h_kv, dh, window = case["R"], case["h_q"], case["h_kv"], case["dh"], case["window"]
    g = h_q // h_kv
    table, cu, lens = s["table"].long(), s["cu"].long(), s["kv_len"].long()
    k, v = (_pages(s, x, table).transpose(1, 2).reshape(R, h_kv, -1, dh)[:, :, :L] for x in ("k", "v"))
    qp, r, i = _padded(s)
    scores = torch.matmul(qp, k.transpose(2, 3).contiguous())
    pos = (lens - (cu[1:] - cu[:-1]))[:, None] + torch.arange(n, device=qp.device)[None, :]  # [R, n]
    j = torch.arange(L, device=qp.device)
    seen = (j[None, None, :] <= pos[:, :, None]) & (j[None, None, :] < lens[:, None, None])
    if window:
        seen &= j[None, None, :] > pos[:, :, None] - window
    scores = scores.reshape(R, h_kv, g, n, L).masked_fill(~seen[:, None, None], float("-inf"))
    w = (scores - scores.amax(-1, keepdim=True).clamp(min=-1e30)).exp()
    w = w / w.sum(-1, keepdim=True).clamp(min=1e-30)
    o = torch.matmul(w.reshape(R, h_kv, g * n, L), v.contiguous()).reshape(R, h_kv, g, n, dh).permute(0, 3, 1, 2, 4).reshape(R, n, h_q, dh)
    return o[r, i].to(s["q"].dtype)


def _plain_shared(s):
    """The prefix once for the tokens of all requests, the rest of each request padded to the longest, one softmax over both."""
    case, n, p = s["case"], s["max_new"], s["case"]["page"]
    R, h_q, h_kv, dh = case["R"], case["h_q"], case["h_kv"], case["dh"]
    g, common, L = h_q // h_kv, case["prefix"] // p, s["max_own"]
    table, cu, lens = s["table"].long(), s["cu"].long(), s["kv_len"].long() - common * p
    qp, r, i = _padded(s)
    pos = (lens - (cu[1:] - cu[:-1]))[:, None] + torch.arange(n, device=qp.device)[None, :]
    j = torch.arange(L, device=qp.device)
    seen = (j[None, None, :] <= pos[:, :, None]) & (j[None, None, :] < lens[:, None, None])
    k, v = (_pages(s, x, table[:, common:]).transpose(1, 2).reshape(R, h_kv, -1, dh)[:, :, :L].contiguous() for x in ("k", "v"))
    mine = torch.matmul(qp, k.transpose(2, 3).contiguous()).reshape(R, h_kv, g, n, L).masked_fill(~seen[:, None, None], float("-inf"))
    mine = mine.reshape(R, h_kv, g * n, L)
    kc, vc = (_pages(s, x, table[0, :common]).transpose(0, 1).reshape(h_kv, -1, dh).contiguous() for x in ("k", "v"))
    every = qp.transpose(0, 1).reshape(h_kv, R * g * n, dh)
    theirs = torch.matmul(every, kc.transpose(1, 2).contiguous())
    if theirs.shape[2] == 0:  # a prefix without a whole page
        top = mine.amax(-1, keepdim=True).clamp(min=-1e30)
    else:
        top = torch.maximum(mine.amax(-1, keepdim=True), theirs.amax(-1).reshape(h_kv, R, g * n, 1).transpose(0, 1)).clamp(min=-1e30)
    w, wc = (mine - top).exp(), (theirs - top.transpose(0, 1).reshape(h_kv, R * g * n, 1)).exp()
    total = w.sum(-1, keepdim=True) + wc.sum(-1).reshape(h_kv, R, g * n, 1).transpose(0, 1)
    o = torch.matmul(w, v) + torch.matmul(wc, vc).reshape(h_kv, R, g * n, dh).transpose(0, 1)
    o = (o / total.clamp(min=1e-30)).reshape(R, h_kv, g, n, dh).permute(0, 3, 1, 2, 4).reshape(R, n, h_q, dh)
    return o[r, i].to(s["q"].dtype)


# ---- what a pass cannot do without --------------------------------------------------


def _size(name):
    return 2 if name == "bf16" else 4


def work(case):
    op, e, dh = case["op"], _size(case["dtype"]), case["dh"]
    if op == "append8":
        T, h_q, h_kv, rot = case["T"], case["h_q"], case["h_kv"], case["rot"]
        return {"bytes": T * ((2 * h_q + 2 * h_kv) * dh * e + 2 * h_kv * (dh + 1) + 4 * rot + 8), "flops": 3 * T * (h_q + h_kv) * rot}
    if op == "read8":
        return {"bytes": case["T"] * (2 * case["h_kv"] * (dh + 1 + dh * e) + 4), "flops": 0}
    ctx, new = _lens(case)
    T, h_q, h_kv = sum(new), case["h_q"], case["h_kv"]
    if op == "attend8":
        row, W = dh + 1, case["window"]
        keys = pairs = 0
        for c, n in zip(ctx, new):
            keys += c + n - (max(0, c + 1 - W) if W else 0)
            full = min(n, max(0, W - c)) if W else n  # tokens that see everything before them
            pairs += _pairs(c, full) + (n - full) * W
    else:
        row = dh + 1 if case["cache"] == "e4m3" else dh * e
        common = case["prefix"] // case["page"] * case["page"]
        over = case["prefix"] - common
        keys = common + sum(over + c + n for c, n in zip(ctx, new))
        pairs = sum(_pairs(case["prefix"] + c, n) for c, n in zip(ctx, new))
    return {"bytes": 2 * keys * h_kv * row + 2 * T * h_q * dh * e, "flops": 4 * pairs * h_q * dh}


# ---- the definitions, in 64 bits ----------------------------------------------------


def exact(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = globals()["_prepare_" + case["op"]](case, g)
    return globals()["_exact_" + case["op"]](case, s)


def _stand_for(codes, b=None):
    """e4m3 by its definition: a sign, four bits of exponent (bias 7, 0 for subnormal), three of significand."""
    c = torch.arange(256, device="cuda", dtype=torch.float64)
    ex, m = (c % 128) // 8, c % 8
    v = torch.where(ex > 0, (8 + m) * 2.0 ** (ex - 10), m * 2.0 ** -9) * torch.where(c < 128, 1.0, -1.0)
    v = v[codes.view(torch.uint8).long()]
    return v if b is None else v * (2.0 ** (b.double() - 127))[..., None]


def _exact_append8(case, s):
    """Codes before their rounding to 8 bits, in units of their row's power of two; the powers' bytes are whole numbers."""
    rot, p = case["rot"], case["page"]
    at = s["pos"].long()
    turn_by = torch.complex(s["rope"][at, : rot // 2].double(), s["rope"][at, rot // 2:].double())[:, None, :]

    def turn(x):
        x = x.double()
        z = torch.complex(x[..., : rot // 2].contiguous(), x[..., rot // 2: rot].contiguous()) * turn_by
        return torch.cat([z.real, z.imag, x[..., rot:]], -1)

    out, slot = {"q_out": turn(s["q"])}, s["slot"].long()
    for n, x in (("k", turn(s["k"])), ("v", s["v"].double())):
        b = torch.ceil(torch.log2(x.abs().amax(-1, keepdim=True) / 448)).clamp(-117, 119)
        flat = _stand_for(s[n + "_cache"]).permute(0, 2, 1, 3).reshape(-1, case["h_kv"], case["dh"])
        flat = flat.index_copy(0, slot, x / 2.0 ** b)
        out[n + "_cache"] = flat.reshape(-1, p, case["h_kv"], case["dh"]).permute(0, 2, 1, 3).contiguous()
    return out


def _exact_read8(case, s):
    slot, out = s["slot"].long(), {}
    for n in ("k", "v"):
        x = _stand_for(s[n + "_cache"], s[n + "_exp"])
        out[n + "_out"] = x.permute(0, 2, 1, 3).reshape(-1, case["h_kv"], case["dh"])[slot]
    return out


def _exact_rows(case, s, name, pages):
    x = s[name + "_cache"][pages].double() if "k_exp" not in s else _stand_for(s[name + "_cache"].view(torch.uint8)[pages], s[name + "_exp"][pages])
    return x.permute(1, 0, 2, 3).reshape(case["h_kv"], -1, case["dh"])


def _exact_requests(case, s, lens, window):
    """Request by request and head by head over the pages in its row of the table."""
    h_kv, g, dh = case["h_kv"], case["h_q"] // case["h_kv"], case["dh"]
    cu, out = s["cu"].tolist(), []
    for r, m in enumerate(lens):
        n = cu[r + 1] - cu[r]
        pages = s["table"][r, : _ceil(m, case["page"])].long()
        k, v = (_exact_rows(case, s, x, pages)[:, :m] for x in ("k", "v"))
        q = s["q"][cu[r]:cu[r + 1]].double().reshape(n, h_kv, g, dh)
        far = torch.arange(m, device=k.device)[None, :] - (m - n + torch.arange(n, device=k.device))[:, None]  # key minus token position
        hidden = torch.where((far > 0) | ((far <= -window) if window else (far > 0)), float("-inf"), 0.0)[:, None, :]
        heads = []
        for h in range(h_kv):
            x = (q[:, h].reshape(n * g, dh) @ k[h].t()).reshape(n, g, m) / dh ** 0.5 + hidden
            heads.append((torch.softmax(x, -1).reshape(n * g, m) @ v[h]).reshape(n, g, dh))
        out.append(torch.stack(heads, 1).reshape(n, case["h_q"], dh))
    return torch.cat(out)


def _exact_attend8(case, s):
    return _exact_requests(case, s, s["kv_len"].tolist(), case["window"])


def _exact_shared(case, s):
    return _exact_requests(case, s, s["kv_len"].tolist(), 0)
