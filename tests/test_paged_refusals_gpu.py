"""Refusals of the paged entry points that come before anything is allocated or launched."""

import pytest

torch = pytest.importorskip("torch")

import online_activation_aware_b200 as ttq

pytestmark = pytest.mark.gpu


def test_too_many_alternatives_are_refused_without_memory_for_them():
    x = torch.zeros(3000, 20000, dtype=torch.bfloat16, device="cuda")
    tokens = torch.zeros(3000, dtype=torch.int64, device="cuda")
    ttq.token_logprobs(x, tokens, 32)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    for top in (33, 20000, 20001, 1 << 40):
        with pytest.raises(ttq.TTQError):
            ttq.token_logprobs(x, tokens, top)
    # log probabilities and entropies of 3000 rows are 24 KB; 33 alternatives of each 1.2 MB
    assert torch.cuda.max_memory_allocated() - before <= 1 << 16
    assert ttq.device_status() == 0
