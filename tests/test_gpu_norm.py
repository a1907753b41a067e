"""Norms of queries and keys with the position rotation, on the GPU against the
formula in 64 bits.

Tolerance. The squares of a head are summed in fp32 in at most 20 roundings of
2^-24, the mean and eps take four more; the root halves that (12 * 2^-24 < 0.75 *
2^-20). The reciprocal root is off by 2^-22, the sine and cosine by 2^-22, the
products with the root and the weight and the rotation's products and sum by five
roundings of 2^-24. In all less than 2^-19 of the sum of a result's products'
sizes, before the one rounding to bf16 (2^-8 of the value; 2^-134, half of the
smallest step, near zero).
"""
import numpy as np
import pytest
import torch

import block_sparse_attention_causal_gb300 as wise
from oracle import cache_oracle as C

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


def _bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).cuda()


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _i32(x):
    return None if x is None else torch.tensor(np.asarray(x).tolist(), dtype=torch.int32).cuda()


def _weights(rng, heads, d, kind, per_head):
    w = torch.from_numpy(1.0 + 0.3 * rng.standard_normal((heads, d) if per_head else (d,))).to(kind).cuda()
    return w, lambda h: _np(w)[h] if per_head else _np(w)


def _want(x, positions, freq, pairs, weight, eps, axes):
    """x [b, heads, n, d]; positions [b][n] or [axes][b][n]."""
    out, size = np.zeros(x.shape), np.zeros(x.shape)
    for b, h, i in np.ndindex(*x.shape[:3]):
        pos = positions[b][i] if axes is None else [p[b][i] for p in positions]
        out[b, h, i], size[b, h, i] = C.norm_rotate(x[b, h, i], pos, freq, pairs, None if weight is None else weight(h), eps, axes)
    return out, size


def _close(got, want, size):
    tol = 2.0 ** -8 * np.abs(want) + (1 + 2.0 ** -8) * 2.0 ** -19 * size + 2.0 ** -134
    off = np.abs(got - want)
    assert np.all(off <= tol), f"{np.max(off - tol):.3e} past the bound"


# (batch, n, heads, kv_heads, d, rotary, pairs, axes, per head, weights of q, k, type, scale of the rows)
ROTATE = [
    (1, 1, 1, 1, 64, 64, False, 1, False, True, True, torch.bfloat16, 1.0),
    (2, 7, 8, 2, 64, 32, True, 1, False, True, True, torch.float32, 1.0),
    (3, 5, 5, 5, 96, 96, False, 3, True, True, True, torch.float32, 3.0),
    (1, 33, 4, 1, 96, 48, True, 2, False, True, False, torch.bfloat16, 1e-4),    # eps counts; keys only rotated
    (2, 9, 2, 6, 96, 0, False, 1, True, False, True, torch.bfloat16, 1.0),       # more keys than queries; no rotation
    (1, 19, 32, 8, 128, 128, False, 1, False, True, True, torch.bfloat16, 100.0),
    (2, 3, 16, 1, 128, 64, True, 3, True, True, True, torch.bfloat16, 1.0),
    (1, 4, 3, 3, 128, 16, False, 4, False, False, False, torch.bfloat16, 1.0),   # neither is normed
    (1, 700, 2, 1, 64, 64, True, 1, False, True, True, torch.bfloat16, 1.0),
]


@pytest.mark.parametrize("case", ROTATE, ids=lambda c: "-".join(str(x) for x in c[:9]))
def test_norm_rotate(case):
    b, n, h, hk, d, rotary, pairs, axes, per_head, with_q, with_k, kind, scale = case
    rng = np.random.default_rng(7)
    # queries and keys side by side, as a projection leaves them
    rows = _bf16(rng.standard_normal((b, n, h + hk, d)) * scale).transpose(1, 2)
    q, k = rows[:, :h], rows[:, h:]
    qw, qf = _weights(rng, h, d, kind, per_head) if with_q else (None, None)
    kw, kf = _weights(rng, hk, d, kind, per_head) if with_k else (None, None)
    freq = [10000.0 ** (-2.0 * i / max(rotary, 1)) for i in range(rotary // 2)]
    where, pos = None, rng.integers(0, 5000, (b, n))
    rope = wise.rope_frequencies(rotary, inv_freq=freq, pairs=pairs)
    if axes > 1:
        where = rng.integers(0, axes, rotary // 2)
        pos = rng.integers(-3, 5000, (axes, b, n))
        rope.axes = _i32(where)
    got = wise.norm_rotate(q, k, q_norm=qw, k_norm=kw, norm_eps=1e-5, positions=_i32(pos), rope=rope)
    wise.check_device()
    for x, y, w in ((q, got[0], qf), (k, got[1], kf)):
        assert y.is_contiguous() and y.shape == x.shape
        _close(_np(y), *_want(_np(x), pos, freq, pairs, w, 1e-5, where))


def test_norm_rotate_defaults_and_outputs():
    rng = np.random.default_rng(3)
    q, k = _bf16(rng.standard_normal((2, 3, 6, 96))), _bf16(rng.standard_normal((2, 1, 6, 96)))
    rope = wise.rope_frequencies(96)
    w = torch.ones(96, device="cuda")
    out = wise.norm_rotate(q, k, q_norm=w, rope=rope)
    pos = np.broadcast_to(np.arange(6), (2, 6))  # token i has position i
    given = torch.empty_like(q), torch.empty_like(k)
    again = wise.norm_rotate(q, k, q_norm=w, rope=rope, positions=_i32(pos), q_out=given[0], k_out=given[1])
    assert again[0] is given[0] and again[1] is given[1]
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])
    alone, none = wise.norm_rotate(q, q_norm=w, rope=rope)
    assert none is None and torch.equal(alone, out[0])
    # one axis named for every pair is no axis at all
    rope.axes = torch.zeros(48, dtype=torch.int32, device="cuda")
    same = wise.norm_rotate(q, k, q_norm=w, rope=rope, positions=_i32(pos[None]))
    assert torch.equal(same[0], out[0]) and torch.equal(same[1], out[1])
    wise.check_device()


def test_sections_of_a_rope():
    rope = wise.rope_frequencies(64, sections=(8, 12, 12))
    assert rope.axes.tolist() == [0] * 8 + [1] * 12 + [2] * 12
    for bad in ((), (16, 17), (40, -8), (16, 15)):
        with pytest.raises(ValueError):
            wise.rope_frequencies(64, sections=bad)


# (lengths, new_len, n, heads (0: without q), kv_heads, d, page, rotary, pairs, axes, per head)
APPEND = [
    ([0], None, 1, 2, 1, 64, 16, 64, False, 1, False),
    ([5, 16, 0], [3, 0, 2], 3, 8, 2, 64, 16, 64, True, 1, False),
    ([14, 31], [40, 13], 40, 5, 5, 96, 32, 48, False, 3, True),
    ([100], None, 9, 0, 4, 128, 64, 128, False, 2, False),
    ([127, 3], [70, 130], 130, 4, 2, 128, 128, 32, True, 1, True),
    ([40], None, 600, 32, 8, 96, 16, 96, True, 3, False),      # four heads ahead
    ([7] * 9, None, 2, 40, 40, 96, 16, 96, False, 1, False),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(str(x) for x in c[2:]))
def test_append_with_norms(case):
    lengths, news, n, h, hk, d, page, rotary, pairs, axes, per_head = case
    rng = np.random.default_rng(11)
    b = len(lengths)
    used = [(x + n + page - 1) // page for x in lengths]
    n_pages = sum(used) + 2
    order = rng.permutation(n_pages)
    table = np.full((b, max(used) + 1), -1, np.int32)
    at = 0
    for s, u in enumerate(used):
        table[s, :u] = order[at:at + u]
        at += u
    rows = _bf16(rng.standard_normal((b, n, h + 2 * hk, d))).transpose(1, 2)
    q, k, v = rows[:, :h] if h else None, rows[:, h:h + hk], rows[:, h + hk:]
    pools = [_bf16(rng.standard_normal((n_pages, hk, page, d))) for _ in range(2)]
    before = [p.clone() for p in pools]
    cache = wise.PagedCache(pools[0], pools[1], _i32(table), _i32(lengths))
    qw, qf = _weights(rng, h, d, torch.float32, per_head) if h else (None, None)
    kw, kf = _weights(rng, hk, d, torch.float32, per_head)
    freq = [50000.0 ** (-2.0 * i / rotary) for i in range(rotary // 2)]
    rope = wise.rope_frequencies(rotary, inv_freq=freq, pairs=pairs)
    where, pos, given = None, [[x + i for i in range(n)] for x in lengths], None
    if axes > 1:
        where, pos = rng.integers(0, axes, rotary // 2), rng.integers(0, 100000, (axes, b, n))
        rope.axes, given = _i32(where), _i32(pos)
    got = wise.cache_append(cache, k, v, q=q, new_len=_i32(news), positions=given, rope=rope, q_norm=qw, k_norm=kw)
    wise.check_device()
    want, size = _want(_np(k), pos, freq, pairs, kf, 1e-6, where)
    kp, vp = _np(before[0]), _np(before[1])
    ks = np.zeros(kp.shape)
    for s in range(b):
        for i in range(n if news is None else news[s]):
            pg, row = C.slot(table, s, lengths[s] + i, page)
            kp[pg, :, row], ks[pg, :, row], vp[pg, :, row] = want[s, :, i], size[s, :, i], _np(v)[s, :, i]
    untouched = ks == 0
    assert np.array_equal(_np(cache.k_pages)[untouched], _np(before[0])[untouched])
    _close(_np(cache.k_pages)[~untouched], kp[~untouched], ks[~untouched])
    assert np.array_equal(_np(cache.v_pages), vp)
    if h:
        _close(_np(got), *_want(_np(q), pos, freq, pairs, qf, 1e-6, where))


def test_append_without_norms_but_axes_matches_the_plain_append():
    """Axes that all carry the same positions rotate as one does."""
    rng = np.random.default_rng(5)
    x = [_bf16(rng.standard_normal((2, 4, 21, 128))) for _ in range(3)]
    table, lengths = _i32([[0, 1, 2], [3, 4, 5]]), _i32([10, 3])
    out = []
    for axes in (False, True):
        pools = [torch.zeros((6, 4, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        cache = wise.PagedCache(pools[0], pools[1], table, lengths)
        pos = _i32(rng.integers(0, 9, (2, 21))) * 0 + lengths[:, None] + torch.arange(21, dtype=torch.int32, device="cuda")
        rope = wise.rope_frequencies(128, sections=(20, 20, 24) if axes else None)
        q = wise.cache_append(cache, x[0], x[1], q=x[2], rope=rope,
                              positions=pos[None].expand(3, 2, 21).contiguous() if axes else pos.contiguous())
        out.append((q, *pools))
    wise.check_device()
    for a, b in zip(*out):
        off = (a.float() - b.float()).abs()
        # the two kernels may contract products differently: one more rounding to bf16 at most
        assert torch.all(off <= 2.0 ** -7 * a.float().abs() + 2.0 ** -19)


def test_zero_rows_and_large_ones():
    q = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16, device="cuda")
    q[0, 1] = 2.0 ** 50
    w = torch.full((64,), 0.5, device="cuda")
    out, _ = wise.norm_rotate(q, q_norm=w)
    assert torch.all(out[0, 0] == 0) and torch.all(out[0, 1] == 0.5)


def test_bad_entries_are_flagged_and_skipped():
    q = _bf16(np.random.default_rng(1).standard_normal((1, 2, 4, 64)))
    w = torch.ones(64, device="cuda")
    rope = wise.rope_frequencies(64, sections=(16, 16))
    pos = torch.arange(8, dtype=torch.int32, device="cuda").reshape(2, 1, 4)
    good, _ = wise.norm_rotate(q, q_norm=w, rope=rope, positions=pos)
    wise.check_device()
    rope.axes[3] = 2
    rope.axes[7] = -1
    out, _ = wise.norm_rotate(q, q_norm=w, rope=rope, positions=pos)
    with pytest.raises(wise.WiseError):
        wise.check_device()
    plain, _ = wise.norm_rotate(q, q_norm=w)
    for i in range(32):
        ref = plain if i in (3, 7) else good
        assert torch.equal(out[..., i], ref[..., i]) and torch.equal(out[..., 32 + i], ref[..., 32 + i])
    # tokens past the table, a page outside the pool, a negative length
    pools = [torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for table, lengths in (([[0, 1]], [30]), ([[0, 4]], [15]), ([[0, -1]], [15]), ([[0, 1]], [-2])):
        cache = wise.PagedCache(pools[0], pools[1], _i32(table), _i32(lengths))
        for p in pools:
            p.zero_()
        wise.cache_append(cache, q, q, k_norm=w)
        with pytest.raises(wise.WiseError):
            wise.check_device()
        written = [int((p.abs().sum((1, 3)) > 0).sum()) for p in pools]
        room = max(0, min(len(table[0]) * 16, 16 if table[0][1] not in (1,) else 32) - lengths[0]) if lengths[0] >= 0 else 0
        assert written == [min(4, room)] * 2
