"""The example that serves a small decoder with sparse drafts, dense verification and
rollback: its sequences and logits against a float64 decoder without cache or drafts."""

import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle
from oracle import serving as S
from tests.helpers import say

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    spec = importlib.util.spec_from_file_location("draft_and_verify", os.path.join(ROOT, "examples", "draft_and_verify.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def f64(t):
    return t.double().cpu().numpy()


def full_logits(model, seq):
    """The full model's logits at every position of one sequence, in float64."""
    h = f64(model.embed)[seq]
    n, h_q, h_kv, dh = len(seq), model.h_q, model.h_kv, model.dh
    x = S.rms_norm(h, f64(model.first.w_pre), 1e-5)
    lo, hi = S.seen(n, n, 0)
    rope = model.rope.cpu().numpy()
    for layer in model.layers:
        qkv = (x @ f64(layer["qkv"]).T).reshape(n, h_q + 2 * h_kv, dh)
        q, k = (S.rotate(t, np.arange(n), rope, dh) for t in (qkv[:, :h_q], qkv[:, h_q:h_q + h_kv]))
        a = S.attend(q, k, qkv[:, h_q + h_kv:], lo, hi, dh ** -0.5)[0].reshape(n, -1)
        h, x = S.residual_norm(h, a @ f64(layer["out"]).T, f64(layer["before_ffn"].w_pre))
        ffn = layer["ffn"]
        y = oracle.dense_chunk(f64(ffn.w_gate), f64(ffn.w_up), f64(ffn.w_down_t), x)
        h, x = S.residual_norm(h, y, f64(layer["after_ffn"].w_pre))
    return x @ f64(model.head).T


def test_prompt_chunk_and_single_token_logits_match_float64():
    """The same sequence fed as a prompt, as single tokens, and as a prompt, a chunk and a rolled
    back chunk. fp32 layers: some twenty products and norms in a row, each off by at most
    8 u sqrt(688) = 1.3e-5 of its size, with a gain of a few through the norms."""
    m = load()
    g = np.random.default_rng(0)
    seqs = [g.integers(0, 500, n).tolist() for n in (40, 23, 57)]
    want = [full_logits(m.Decoder(), s) for s in seqs]

    def off(got, r, lo, hi):
        ref = want[r][lo:hi]
        return np.abs(got - ref).max() / np.abs(ref).max()

    model = m.Decoder()
    got = model.step(seqs, [0, 0, 0], dense=True)
    cu = model.cu.tolist()
    errs = [off(f64(got[cu[r]:cu[r + 1]]), r, 0, len(seqs[r])) for r in range(3)]
    say(f"[example] prompt {errs}")
    model = m.Decoder()
    model.step([s[:10] for s in seqs], [0, 0, 0], dense=True)
    model.step([s[-16:] for s in seqs], [10, 7, 10], dense=True)  # tokens that are not the sequence's: rolled back
    got = model.step([seqs[0][10:26], [], seqs[2][10:11]], [10, 10, 10], dense=True)
    errs += [off(f64(got[:16]), 0, 10, 26), off(f64(got[16:]), 2, 10, 11)]
    for i in range(12):  # single tokens, one request ahead of another
        got = model.step([seqs[0][26 + i:27 + i], seqs[1][10 + i:11 + i], seqs[2][11 + i:12 + i]], [26 + i, 10 + i, 11 + i], dense=True)
        errs += [off(f64(got[r:r + 1]), r, p, p + 1) for r, p in enumerate((26 + i, 10 + i, 11 + i))]
    say(f"[example] worst of chunks and single tokens {max(errs)}")
    assert max(errs) < 1e-3


@pytest.mark.parametrize("sparsity,draft", [(0.5, 16), (0.9, 5), (0.0, 16)])
def test_drafts_never_change_the_sequence(sparsity, draft):
    """Whatever is drafted, the sequences are the full model's greedy ones (the float64 decoder's,
    except where its two best logits are closer than the fp32 error); drafts of the full
    model itself (sparsity 0) are all kept but for the chunk's end."""
    m = load()
    model = m.Decoder(sparsity=sparsity, requests=2)
    prompts = [[3, 1, 4, 1, 5], list(range(30, 47))]
    seqs, kept, drafted = model.generate(prompts, 24, draft)
    say(f"[example] sparsity {sparsity} draft {draft}: kept {kept} of {drafted}")
    assert model.status.item() == 0
    for p, s in zip(prompts, seqs):
        assert len(s) == len(p) + 24 and s[:len(p)] == p
        ref = full_logits(model, s)
        for i in range(len(p), len(s)):
            row = ref[i - 1]
            assert row[s[i]] >= row.max() - 2e-3 * np.abs(ref).max(), (i, s[i], row.argmax())
    if sparsity == 0.0:
        assert kept >= drafted - 2 * 15 - 2
    if sparsity == 0.9:
        assert kept < drafted  # drafts were dropped, so the rollback was at work


def test_pages_come_back():
    """After ending every request (nothing kept, nothing new) all pages are free again."""
    m = load()
    model = m.Decoder(requests=3)
    model.generate([[1], [2, 3], list(range(40))], 20)
    assert 0 < model.n_free.item() < model.free.numel()
    from contextual_activation_sparsity_amd import binding as B

    z = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    B.kv_cache_plan(model.layers[0]["cache"], torch.tensor(model.held, dtype=torch.int32, device="cuda"), z(3), z(3), model.table,
                    model.free, model.n_free, model.n_free_next, model.cu, model.kv_len, z(1), z(1), model.status)
    assert model.status.item() == 0 and model.n_free_next.item() == model.free.numel()
    assert sorted(model.free.tolist()) == list(range(model.free.numel()))


def test_command_runs(capsys):
    load().main(["--requests", "2", "--tokens", "20"])
    out = capsys.readouterr().out
    assert "2 requests, 20 tokens each" in out and "pages free" in out
