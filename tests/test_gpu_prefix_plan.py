"""The word that orders a shared-prefix call's own parts behind its plan: each
call writes it, reads it and takes it back, whatever its workspace held before.
Results are compared bit for bit with the first call's."""
import pytest
import torch

import block_sparse_attention_causal_gb300 as wise
from block_sparse_attention_causal_gb300 import _lib

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


def _batch(b, h, hk, n, d, page, prefix, own, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    whole, cols = prefix // page, (own + n) // page + 2
    table = torch.empty((b, whole + cols), dtype=torch.int32, device="cuda")
    table[:, :whole] = torch.arange(whole, device="cuda")
    table[:, whole:] = whole + torch.arange(b * cols, device="cuda").reshape(b, cols)
    k, v = (torch.randn((whole + b * cols, hk, page, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    lengths = prefix + torch.randint(0, own, (b,), generator=g, device="cuda").to(torch.int32)
    q = torch.randn((b, h, n, d), generator=g, device="cuda").to(torch.bfloat16)
    return wise.PagedCache(k, v, table, lengths), q, torch.tensor([prefix], dtype=torch.int32, device="cuda")


# narrow and wide units in either part; a batch that shares nothing
@pytest.mark.parametrize("b,h,hk,n,d,prefix", [(6, 8, 2, 1, 64, 512), (8, 8, 2, 6, 96, 640), (3, 4, 1, 40, 128, 1024),
                                               (5, 4, 1, 20, 64, 128), (4, 8, 2, 1, 128, 0)])
def test_the_plan_s_word_is_this_call_s(b, h, hk, n, d, prefix):
    cache, q, pre = _batch(b, h, hk, n, d, 32, prefix, 300, seed=b)
    size = _lib.load().wise_attn_prefix_workspace(wise._check_cache(cache)[0], h, n, 1)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    assert ws.data_ptr() % 256 == 0
    want = wise.prefix_attention(q, cache, pre, out_dtype=torch.float32, workspace=ws)
    wise.check_device()
    assert not ws[:8].any(), "a later call could take the word for its own"
    g = torch.Generator(device="cuda").manual_seed(1)
    left = ws.clone()
    for fill in (lambda: ws.fill_(255), lambda: ws.random_(0, 256, generator=g), lambda: ws.copy_(left), lambda: ws.zero_(), lambda: None):
        fill()
        got = wise.prefix_attention(q, cache, pre, out_dtype=torch.float32, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and not ws[:8].any()
    wise.check_device()


def test_one_workspace_for_calls_of_different_shapes():
    """Calls in turn through one workspace, their words at the same place and the
    rest of their plans at others."""
    forms = [_batch(6, 8, 2, 1, 64, 32, 512, 300, 1), _batch(3, 4, 1, 40, 128, 32, 1024, 200, 2), _batch(5, 4, 1, 20, 64, 32, 128, 90, 3)]
    size = max(_lib.load().wise_attn_prefix_workspace(wise._check_cache(c)[0], q.shape[1], q.shape[2], 1) for c, q, _ in forms)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    want = [wise.prefix_attention(q, c, p) for c, q, p in forms]
    torch.cuda.synchronize()
    for _ in range(30):
        for (c, q, p), w in zip(forms, want):
            got = wise.prefix_attention(q, c, p, workspace=ws)
            assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [wise.prefix_attention(q, c, p, workspace=ws) for c, q, p in forms]
    for _ in range(20):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x[0], w[0]) and torch.equal(x[1], w[1]) for x, w in zip(got, want)) and not ws[:8].any()
    wise.check_device()
