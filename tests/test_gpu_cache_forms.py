"""The paged-cache operators on the GPU in the forms that differ in code:
rotations at every size of angle, every instance of the attention kernels, pages
outside the pool under each of them, long prompts and long accepted paths.

Tolerances. A rounding to bf16 is off by at most 2^-8 of the value, one in fp32
by 2^-24.
 * rotation: the sine and cosine are good to 2^-22 of their value; the two
   products and their sum add 2^-24 each, so a result is off by less than 2^-21
   of |x cos a| + |y sin a| before its one rounding to bf16 (times 1 + 2^-21).
"""
import math

import numpy as np
import pytest
import torch

import block_sparse_attention_causal_gb300 as wise

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

BF16, F32 = 2.0 ** -8, 2.0 ** -24


def _bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


def _np(t):
    return t.double().cpu().numpy()


def _i32(x):
    return None if x is None else torch.tensor(np.asarray(x).tolist(), dtype=torch.int32).cuda()


def _steps(freq):
    return [int(round(f / (2.0 * math.pi) * 2.0 ** 64)) % (1 << 64) for f in freq]


def _turn(step, position):
    """(cos, sin) of position * step / 2^64 turns: quarter turns taken off as
    whole numbers, so that small values keep their bits."""
    at = (step * int(position) + (1 << 61)) % (1 << 64)
    rest = (at % (1 << 62) - (1 << 61)) * math.pi * 2.0 ** -63
    c, s = math.cos(rest), math.sin(rest)
    return [(c, s), (-s, c), (-c, -s), (s, -c)][at >> 62]


# ----------------------------------------------------------------- rotation

@pytest.mark.parametrize("pairs", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("base", [1e4, 5e5, 1e8])
def test_small_sines_and_cosines_keep_their_bits(base, pairs):
    """Pairs (x, 0), (0, y) and (x, y) at small angles, at angles next to every
    quarter turn and at far positions: each value to its own rounding."""
    d, page = 128, 16
    freq = [base ** (-2.0 * i / d) for i in range(d // 2)]
    freq[-1], freq[-2], freq[-3] = 2.0 * math.pi / 4.0, 2.0 * math.pi / 8.0, 2.0 * math.pi / 4.0 + 1e-9
    rope = wise.rope_frequencies(d, inv_freq=freq, pairs=pairs)
    pos = [0, 1, 2, 3, 5, 7, 100, 12345, 10 ** 6 + 1, 2 ** 30 + 3, 2 ** 31 - 1, -1, -7]
    n = len(pos)
    x, y = np.zeros((3, n, d // 2)), np.zeros((3, n, d // 2))
    rng = np.random.default_rng(int(base))
    x[0], y[1] = 1.0, -1.5
    x[2], y[2] = _np(_bf16(rng.standard_normal((n, d // 2)))), _np(_bf16(rng.standard_normal((n, d // 2)) * 1e-3))
    k = np.zeros((1, 3, n, d))
    a, b = (slice(0, None, 2), slice(1, None, 2)) if pairs else (slice(0, d // 2), slice(d // 2, None))
    k[0, ..., a], k[0, ..., b] = x, y
    pool = torch.zeros((1, 3, page, d), dtype=torch.bfloat16, device="cuda")
    cache = wise.PagedCache(pool, torch.zeros_like(pool), _i32([[0]]), _i32([0]))
    kt = _bf16(k).cuda()
    q = wise.cache_append(cache, kt, kt, q=kt, positions=_i32([pos]), rope=rope)
    wise.check_device()
    cs = np.array([[_turn(s, t) for s in _steps(freq)] for t in pos])
    c, s = cs[..., 0], cs[..., 1]
    for got in (_np(cache.k_pages)[0, :, :n], _np(q)[0]):
        for part, u, v in ((a, x * c, -y * s), (b, y * c, x * s)):
            want, size = u + v, np.abs(u) + np.abs(v)
            assert np.all(np.abs(got[..., part] - want) <= BF16 * np.abs(want) + (1 + BF16) * 2.0 ** -21 * size)


# ---------------------------------------------------------- buffers that meet

def test_append_refuses_results_over_its_buffers_and_takes_those_between():
    b, h, hk, n, d, page = 2, 2, 1, 5, 64, 16
    g = torch.Generator(device="cuda").manual_seed(5)
    # one arena: the first sequence's rows, room for the rotated queries, the second's
    rows, room = n * (h + 2 * hk) * d, b * h * n * d
    arena = torch.randn((2 * (rows + room),), generator=g, device="cuda").bfloat16()
    qkv = arena.as_strided((b, n, h + 2 * hk, d), (rows + room, (h + 2 * hk) * d, d, 1)).transpose(1, 2)
    q, k, v = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
    rope = wise.rope_frequencies(d)

    def cache():
        pool = torch.zeros((2, hk, page, d), dtype=torch.bfloat16, device="cuda")
        return wise.PagedCache(pool, pool.clone(), _i32([[0], [1]]), _i32([3, 0]))
    plain, given = cache(), cache()
    before = qkv.clone()
    want = wise.cache_append(plain, k, v, q=q, rope=rope)
    between = arena[rows:rows + room].view(b, h, n, d)
    got = wise.cache_append(given, k, v, q=q, q_out=between, rope=rope)
    assert got is between and torch.equal(got, want) and torch.equal(qkv, before)
    assert torch.equal(plain.k_pages, given.k_pages) and torch.equal(plain.v_pages, given.v_pages)
    for off in (0, rows - 8, rows + 8):
        with pytest.raises(wise.WiseError):
            wise.cache_append(given, k, v, q=q, q_out=arena[off:off + room].view(b, h, n, d), rope=rope)
    dense = q.contiguous()
    with pytest.raises(wise.WiseError):
        wise.cache_append(given, k, v, q=dense, q_out=dense, rope=rope)
    with pytest.raises(wise.WiseError):
        wise.cache_append(given, k, v, q=q, q_out=given.k_pages.view(-1)[:room].view(b, h, n, d), rope=rope)
    wise.check_device()
    assert torch.equal(qkv, before) and torch.equal(plain.k_pages, given.k_pages)
