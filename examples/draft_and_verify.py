#!/usr/bin/env python3
"""A small decoder served with the library: sparse drafts, dense verification, rollback.

    python examples/draft_and_verify.py [--requests 3] [--tokens 48] [--draft 16] [--cache own|e4m3]

Several requests are decoded greedily at once ("SIRIUS: Contexual Sparisty with Correction
for Efficient LLMs", Approach). Each period drafts up to 16 tokens a request with the sparse
FFN (``sparse_ffn_decode``, one token of up to four requests a step), then runs the drafted
chunk through the full layers (``ffn_dense_chunk``), keeps the tokens on which both agree and
one of the full model's own, and drops the rest. The paged cache carries this: the plan takes
pages for new tokens and gives back those of dropped ones, ``kv_cache_append`` rewrites the
drafted positions with the full model's keys and values, ``kv_cache_attend`` serves single
tokens, chunks and prompts alike, and ``residual_norm`` stands between all blocks; with ``--cache e4m3``
the cache holds 8 bits a value (the ``kv8_cache`` calls). Weights are random (so the agreement
means nothing beyond showing the mechanism); the projections are plain torch products.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from contextual_activation_sparsity_amd import binding as B  # noqa: E402


class Decoder:
    """Layers, their caches, and the bookkeeping of one batch of requests."""

    def __init__(self, layers=2, d=256, f=688, h_q=4, h_kv=2, dh=64, vocab=500, requests=3, max_len=256, page=16,
                 sparsity=0.5, dtype=torch.float32, seed=0, cache="own"):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rnd = lambda *s, std: (torch.randn(s, generator=g, device="cuda") * std).to(dtype)  # noqa: E731
        self.d, self.h_q, self.h_kv, self.dh, self.R, self.dtype, self.max_len = d, h_q, h_kv, dh, requests, dtype, max_len
        self.embed, self.head = rnd(vocab, d, std=1.0), rnd(vocab, d, std=1.0)
        self.layers = []
        cols = -(-max_len // page)
        n_pages = requests * cols
        for _ in range(layers):
            if cache == "e4m3":
                k, v = (torch.zeros((n_pages, h_kv, page, dh), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
                kv = B.KVCache8(k, v, *(torch.zeros((n_pages, h_kv, page), dtype=torch.uint8, device="cuda") for _ in range(2)), dtype)
            else:
                kv = B.KVCache(*(torch.zeros((n_pages, h_kv, page, dh), dtype=dtype, device="cuda") for _ in range(2)))
            ffn = B.FFNLayer(rnd(f, d, std=d ** -0.5), rnd(f, d, std=d ** -0.5), rnd(f, d, std=f ** -0.5))
            self.layers.append(dict(
                qkv=rnd(h_q * dh + 2 * h_kv * dh, d, std=d ** -0.5), out=rnd(d, h_q * dh, std=(h_q * dh) ** -0.5), ffn=ffn, cache=kv,
                before_ffn=B.ResidualNorm(1 + rnd(d, std=0.1)), after_ffn=B.ResidualNorm(1 + rnd(d, std=0.1)),
                threshold=torch.empty(1, device="cuda")))
        self.first = B.ResidualNorm(1 + rnd(d, std=0.1))
        ang = torch.arange(max_len, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, dh, 2, device="cuda") / dh)[None]
        self.rope = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
        self.append, self.attend, attend_size = (
            (B.kv8_cache_append, B.kv8_cache_attend, B.kv8_cache_attend_workspace_size) if cache == "e4m3" else
            (B.kv_cache_append, B.kv_cache_attend, B.kv_cache_attend_workspace_size))
        # one workspace serves every call: they run in order on one stream
        ffn = self.layers[0]["ffn"]
        self.ws = B.workspace(max(B.sparse_ffn_workspace_size(ffn, 256), attend_size(
            self.layers[0]["cache"], requests, requests * max_len, h_q, max_len, max_len)))
        x = rnd(256, d, std=1.0)
        for layer in self.layers:  # the sparse FFN's thresholds, from tokens of the norm's scale
            B.sparse_ffn_calibrate(layer["ffn"], x, sparsity, layer["threshold"], self.ws)
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.table, self.free = i32(requests, cols), torch.arange(n_pages, dtype=torch.int32, device="cuda")
        self.n_free, self.n_free_next = torch.full((1,), n_pages, dtype=torch.int32, device="cuda"), i32(1)
        self.cu, self.kv_len, self.status = i32(requests + 1), i32(requests), i32(1)
        self.held = [0] * requests  # tokens whose pages the table holds

    def step(self, tokens, keep, dense):
        """Runs tokens[r] (a list for each request) after the first keep[r] tokens of request r;
        returns the logits of all of them, one request after the other."""
        new = [len(t) for t in tokens]
        if max(k + n for k, n in zip(keep, new)) > self.max_len:
            raise ValueError(f"a sequence of more than max_len = {self.max_len} tokens, drafts counted")
        T = sum(new)
        dev = lambda v, dt=torch.int32: torch.tensor(v, dtype=dt, device="cuda")  # noqa: E731
        pos, slot = (torch.empty(T, dtype=torch.int32, device="cuda") for _ in range(2))
        B.kv_cache_plan(self.layers[0]["cache"], dev(self.held), dev(keep), dev(new), self.table, self.free, self.n_free,
                        self.n_free_next, self.cu, self.kv_len, pos, slot, self.status)
        self.n_free, self.n_free_next = self.n_free_next, self.n_free
        self.held = [k + n for k, n in zip(keep, new)]
        h = self.embed[dev([t for one in tokens for t in one], torch.long)]
        x, q, a = torch.empty_like(h), *(torch.empty((T, self.h_q, self.dh), dtype=self.dtype, device="cuda") for _ in range(2))
        y = torch.empty((T, self.d), dtype=torch.float32, device="cuda")
        B.residual_norm(self.first, h, None, None, x)
        for layer in self.layers:
            qkv = (x @ layer["qkv"].t()).view(T, self.h_q + 2 * self.h_kv, self.dh)
            self.append(layer["cache"], qkv[:, self.h_q:-self.h_kv], qkv[:, -self.h_kv:], slot, q=qkv[:, :self.h_q],
                        q_out=q, pos=pos, rope=self.rope)
            self.attend(layer["cache"], q, self.table, self.cu, self.kv_len, a, self.ws, max(max(new), 1), self.max_len)
            B.residual_norm(layer["before_ffn"], h, a.view(T, -1) @ layer["out"].t(), h, x)
            at = B.SFN_MAX_CHUNK if dense else B.SFN_MAX_BATCH
            for i in range(0, T, at):
                if dense:
                    B.ffn_dense_chunk(layer["ffn"], x[i:i + at], y[i:i + at], self.ws)
                else:
                    B.sparse_ffn_decode(layer["ffn"], x[i:i + at], layer["threshold"], self.ws, y=y[i:i + at])
            B.residual_norm(layer["after_ffn"], h, y, h, x)
        return x.float() @ self.head.float().t()

    def generate(self, prompts, n_tokens, draft=16):
        """Greedy decoding of up to n_tokens more a request; returns the sequences and how many
        drafted tokens were kept, of how many."""
        seqs = [list(p) for p in prompts]
        goal = [len(p) + n_tokens for p in prompts]
        logits = self.step(seqs, [0] * self.R, dense=True)
        nxt = logits[self.cu[1:].long() - 1].argmax(-1).tolist()  # after each prompt's last token
        drafted = kept = 0
        while any(len(s) < g for s, g in zip(seqs, goal)):
            live = [len(s) < g for s, g in zip(seqs, goal)]
            base = [len(s) for s in seqs]
            chunk = [[t] if on else [] for t, on in zip(nxt, live)]  # the full model's token opens each chunk
            for i in range(min(draft, B.SFN_MAX_CHUNK) - 1):
                logits = self.step([c[i:] for c in chunk], [b + min(i, len(c)) for b, c in zip(base, chunk)], dense=False)
                for c, t in zip([c for c in chunk if c], logits.argmax(-1).tolist()):
                    c.append(t)
            # the same positions again with the full layers: their keys and values replace the drafts'
            truth = self.step(chunk, base, dense=True).argmax(-1).tolist()
            cu = self.cu.tolist()
            for r, c in enumerate(chunk):
                if not c:
                    continue
                t = truth[cu[r]:cu[r + 1]]
                ok = 1
                while ok < len(c) and c[ok] == t[ok - 1]:
                    ok += 1
                ok = min(ok, goal[r] - base[r])
                seqs[r] += c[:ok]
                nxt[r] = t[ok - 1]
                drafted, kept = drafted + len(c) - 1, kept + ok - 1
        return seqs, kept, drafted


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=3, choices=range(1, B.SFN_MAX_BATCH + 1))
    ap.add_argument("--tokens", type=int, default=48)
    ap.add_argument("--draft", type=int, default=16)
    ap.add_argument("--cache", choices=("own", "e4m3"), default="own")
    a = ap.parse_args(argv)
    model = Decoder(requests=a.requests, dtype=torch.bfloat16, max_len=64 + a.tokens + 16, cache=a.cache)
    prompts = [[(7 * r + 3 * i) % 500 for i in range(5 + 11 * r)] for r in range(a.requests)]
    seqs, kept, drafted = model.generate(prompts, a.tokens, a.draft)
    print(f"{a.requests} requests, {a.tokens} tokens each: {kept} of {drafted} drafted tokens kept; "
          f"{model.n_free.item()} of {model.free.numel()} pages free")
    for p, s in zip(prompts, seqs):
        print(f"  {len(p)} + {s[len(p):][:12]} ...")


if __name__ == "__main__":
    main()
