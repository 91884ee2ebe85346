"""The example that serves a small decoder, with its cache in 8 bits."""

import pytest
import torch

from tests.test_gpu_draft_and_verify import load

pytestmark = pytest.mark.gpu


def test_command_runs(capsys):
    load().main(["--requests", "2", "--tokens", "20", "--cache", "e4m3"])
    assert "2 requests, 20 tokens each" in capsys.readouterr().out


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logits_are_near_those_of_the_models_own_cache(dtype):
    """One prompt of each request through both caches, the same weights. A value in the cache is
    off by up to 2^-4 of itself; this shows that the example hands the right arrays to the right
    calls, no more: the logits of unrelated caches would be uncorrelated."""
    m = load()
    prompts = [[(7 * r + 3 * i) % 500 for i in range(9 + 11 * r)] for r in range(3)]
    own, in8 = (m.Decoder(dtype=dtype, cache=c).step(prompts, [0] * 3, dense=True) for c in ("own", "e4m3"))
    assert torch.isfinite(in8).all() and in8.shape == own.shape
    assert torch.corrcoef(torch.stack([own.flatten(), in8.flatten()]))[0, 1] > 0.9
    assert not torch.equal(own, in8)


def test_pages_come_back():
    """After ending every request all pages are free again: the plan takes the 8-bit cache."""
    m = load()
    model = m.Decoder(requests=3, cache="e4m3")
    seqs, kept, drafted = model.generate([[1], [2, 3], list(range(40))], 20)
    assert [len(s) >= n + 20 for s, n in zip(seqs, (1, 2, 40))] == [True] * 3 and 0 <= kept <= drafted
    assert 0 < model.n_free.item() < model.free.numel()
    from contextual_activation_sparsity_amd import binding as B

    z = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    B.kv_cache_plan(model.layers[0]["cache"], torch.tensor(model.held, dtype=torch.int32, device="cuda"), z(3), z(3), model.table,
                    model.free, model.n_free, model.n_free_next, model.cu, model.kv_len, z(1), z(1), model.status)
    assert model.status.item() == 0 and model.n_free_next.item() == model.free.numel()
    assert sorted(model.free.tolist()) == list(range(model.free.numel()))
