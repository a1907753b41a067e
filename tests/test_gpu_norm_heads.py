"""Norms with rotation at the greatest number of heads that a call takes (queries
and keys together 2^18), weights of every head's own, against the formula in 64
bits: a result is off by 2^-8 of itself and 2^-19 of its two products' sizes."""
import pytest
import torch

import block_sparse_attention_causal_gb300 as wise

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


@pytest.mark.parametrize("d,n,dtype", [(64, 1, torch.float32), (96, 3, torch.bfloat16), (128, 2, torch.float32)])
def test_the_most_heads(d, n, dtype):
    hk = 21
    heads = (1 << 18) - hk
    g = torch.Generator(device="cuda").manual_seed(d)
    q = torch.randn((1, heads, n, d), generator=g, device="cuda").to(torch.bfloat16)
    k = torch.randn((1, hk, n, d), generator=g, device="cuda").to(torch.bfloat16)
    qn, kn = ((torch.rand((m, d), generator=g, device="cuda") + 0.5).to(dtype) for m in (heads, hk))
    rope = wise.rope_frequencies(d)
    got = wise.norm_rotate(q, k, q_norm=qn, k_norm=kn, rope=rope)
    wise.check_device()
    angle = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(d // 2, device="cuda", dtype=torch.float64) * 2 / d)
    cos, sin = torch.cos(angle), torch.sin(angle)
    for x, w, y in ((q, qn, got[0]), (k, kn, got[1])):
        x = x.double()
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.double()[None, :, None]
        a, b = x[..., :d // 2], x[..., d // 2:]
        want = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        size = torch.cat([(a * cos).abs() + (b * sin).abs(), (b * cos).abs() + (a * sin).abs()], -1)
        assert torch.all((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -19 * size)
    with pytest.raises(wise.WiseError):
        wise.norm_rotate(torch.cat([q, q[:, :1]], 1), k)
