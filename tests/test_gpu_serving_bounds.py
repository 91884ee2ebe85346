"""The paged cache's calls at their bounds on the GPU: workspaces of a program's largest step,
lengths past the bounds, counts that do not fit, splits up to the most there are."""

import numpy as np
import pytest
import torch

from oracle import serving as S
from tests.helpers import say
from tests.serving_helpers import attend_oracle, f64, random_cache, within
from tests.test_gpu_draft_and_verify import full_logits, load
from tests.test_gpu_kv_cache import check_attend, i32, run_attend, run_plan

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from contextual_activation_sparsity_amd import binding as B

BF, F32 = torch.bfloat16, torch.float32


def test_one_workspace_for_long_sequences_serves_every_step():
    """The example's workspace is sized for its longest prompts; its single tokens and chunks,
    whose keys are split where a prompt's are not, have to fit into it. The bound is the one of
    test_prompt_chunk_and_single_token_logits_match_float64."""
    m = load()
    model = m.Decoder(max_len=4080)
    g = np.random.default_rng(1)
    seqs = [g.integers(0, 500, n).tolist() for n in (50, 31, 44)]
    want = [full_logits(model, s) for s in seqs]
    say("[example] long bounds")
    model.step([s[:20] for s in seqs], [0, 0, 0], dense=True)
    chunk = f64(model.step([s[20:30] for s in seqs], [20, 20, 20], dense=True))
    one = f64(model.step([s[30:31] for s in seqs], [30, 30, 30], dense=True))
    assert model.status.item() == 0
    for r in range(3):
        top = np.abs(want[r]).max()
        assert np.abs(chunk[10 * r:10 * r + 10] - want[r][20:30]).max() < 1e-3 * top
        assert np.abs(one[r] - want[r][30]).max() < 1e-3 * top
