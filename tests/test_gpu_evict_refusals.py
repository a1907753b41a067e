"""Refusals of eviction that must not cost memory first."""
import pytest
import torch

import block_sparse_attention_causal_gb300 as wise

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


@pytest.mark.parametrize("budget", [65, 1 << 20, (1 << 31) - 1])
def test_a_budget_past_the_new_pages_is_refused_before_anything_is_allocated(budget):
    """Four pages of 16 tokens take 64: more is refused, as an argument, without a
    workspace of the budget's size (1 GB to 4 TB for 512 key heads)."""
    b, hk, page, d = 64, 8, 16, 64
    k, v = (torch.zeros((8 * b, hk, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.arange(8 * b, dtype=torch.int32, device="cuda").reshape(b, 8)
    cache = wise.PagedCache(k, v, table[:, :4].contiguous(), torch.full((b,), 40, dtype=torch.int32, device="cuda"))
    to = table[:, 4:].contiguous()
    weights = torch.rand((b, hk, 64), device="cuda")
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.max_memory_allocated()
    with pytest.raises(wise.WiseError) as e:
        wise.cache_evict(cache, weights, budget, to)
    assert e.value.status == wise._lib.WISE_ERR_INVALID_ARGUMENT
    assert torch.cuda.max_memory_allocated() - before < 1 << 20
    kept, _ = wise.cache_evict(cache, weights, 64, to)  # the most that they take
    wise.check_device()
    assert kept.lengths.tolist() == [40] * b
