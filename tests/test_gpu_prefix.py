"""Attention of batches whose sequences share prefixes, on the GPU against the
formula in 64 bits.

Tolerances are those of the attention over a cache (a score is off by e_s = (d +
8) 2^-24 scale sum |q k|; a weight is rounded to bf16, 2^-8, in the numerator and
in the sum alike; LSE by e_s, 2^-20, and 2^-24 for each addition of the longest
chain and of its value), plus the join of a row's two parts: each part's LSE
off by that bound shifts its share of O by as much, relative to it, and the
join's exponentials and logarithm by 2^-20 more.
"""
import numpy as np
import pytest
import torch

import block_sparse_attention_causal_gb300 as wise
from oracle import cache_oracle as C

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

BF16, F32 = 2.0 ** -8, 2.0 ** -24


def _bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).cuda()


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _i32(x):
    return None if x is None else torch.tensor(np.asarray(x).tolist(), dtype=torch.int32).cuda()


def _shared_cache(rng, starts, prefixes, lengths, news, hk, d, page, scale=1.0):
    """A cache whose sequences name their group's whole shared pages (of the
    first long enough) and hold copies of the tokens of the page in which the
    prefix ends; NaN wherever no token lies."""
    b = len(lengths)
    totals = [x + y for x, y in zip(lengths, news)]
    cols = max(max((t + page - 1) // page for t in totals), 1) + 1
    table = np.full((b, cols), -1, np.int32)
    n_pages = sum((t + page - 1) // page for t in totals) + 3
    free = [int(x) for x in rng.permutation(n_pages)]
    k = np.full((n_pages, hk, page, d), np.nan, np.float32)
    v = k.copy()
    group = [next((g for g in range(len(prefixes)) if starts[g] <= s < starts[g + 1]), None) for s in range(b)]
    first = {}
    for s in range(b):
        p = prefixes[group[s]] if group[s] is not None else 0
        leader = first.get(group[s]) if lengths[s] >= p else None
        whole = p // page if leader is not None else 0
        for c in range((totals[s] + page - 1) // page):
            table[s, c] = table[leader, c] if c < whole else free.pop()
        for t in range(whole * page, totals[s]):
            pg, row = C.slot(table, s, t, page)
            if leader is not None and t < p:
                lp, lr = C.slot(table, leader, t, page)
                k[pg, :, row], v[pg, :, row] = k[lp, :, lr], v[lp, :, lr]
            else:
                k[pg, :, row] = rng.standard_normal((hk, d)) * scale
                v[pg, :, row] = rng.standard_normal((hk, d))
        if group[s] is not None and leader is None and lengths[s] >= p:
            first[group[s]] = s
    return wise.PagedCache(_bf16(k), _bf16(v), _i32(table), _i32(lengths)), table


def _mask(rng, b, n, kind):
    if kind == "run":
        return np.broadcast_to(np.tril(np.ones((n, n), bool)), (b, n, n)).copy(), None
    m = rng.random((b, n, n)) < 0.5
    m[:, n // 2] = False  # a row that sees no new token
    return m, wise.pack_tree_mask(torch.from_numpy(m).cuda())


def _check(q, cache, table, sees, lengths, news, got, dtype):
    o, lse = got
    n, d = q.shape[2], q.shape[3]
    want, want_lse, weight, size = C.tree_attention(_np(q), np.nan_to_num(_np(cache.k_pages)), np.nan_to_num(_np(cache.v_pages)),
                                                    table, lengths, sees, news)
    empty = np.isneginf(want_lse)
    e_s = (d + 8) * F32 * size
    keys = max(x + y for x, y in zip(lengths, news))
    lse_tol = e_s + 2.0 ** -20 + F32 * (64 + keys / 8 + 2 * np.abs(np.where(empty, 0, want_lse)))
    tol = (2 * BF16 + 2 * e_s + 2 * lse_tol + 2.0 ** -19)[..., None] * weight
    tol = tol + (BF16 * np.abs(want) if dtype == torch.bfloat16 else 0.0)
    off = np.abs(_np(o) - want)
    assert np.all(off <= tol), f"O: {np.nanmax(off - tol):.3e} past the bound"
    assert np.all(_np(o)[empty] == 0) and np.all(np.isneginf(_np(lse)[empty]))
    off = np.abs(_np(lse)[~empty] - want_lse[~empty])
    lse_tol = lse_tol + 2.0 ** -20 + F32 * 2 * np.abs(np.where(empty, 0, want_lse))
    assert np.all(off <= lse_tol[~empty]), f"LSE: {np.max(off - lse_tol[~empty]):.3e} past the bound"


# (group starts, prefixes, committed tokens behind the prefix, new_len, n, heads, kv_heads, d, page, mask)
PREFIX = [
    ([0, 2], [128], [0, 1], None, 1, 2, 2, 64, 16, "run"),                         # exactly one tile
    ([0, 3], [127], [5, 0, 9], None, 1, 8, 2, 64, 32, "run"),                      # no whole tile: nothing shared
    ([0, 4], [300], [5, 0, 90, 130], [1, 0, 1, 1], 1, 8, 2, 128, 16, "run"),       # narrow units; a sequence without a token
    ([0, 3], [513], [40, 3, 7], [3, 5, 1], 5, 4, 2, 96, 32, "random"),             # 30 rows
    ([0, 5], [256], [1, 2, 3, 4, 5], None, 3, 8, 2, 64, 64, "random"),             # 60 rows
    ([0, 7], [1000], [10] * 7, None, 4, 8, 2, 128, 128, "run"),                    # 112 rows: streams alternate tiles
    ([0, 8], [640], list(range(8)), None, 6, 8, 2, 96, 16, "random"),              # 192 rows
    ([0, 9], [390], [200, 1, 0, 3, 77, 128, 5, 64, 9], [9, 1, 0, 4, 9, 2, 3, 9, 8], 9, 16, 2, 64, 32, "random"),  # 648 rows
    ([0, 2, 5, 6, 9], [256, 129, 500, 700], [3, 9, 0, 4, 8, 2, 1, 5, 7], None, 2, 4, 1, 128, 64, "run"),  # four groups, one of a single
    ([1, 4, 4, 7], [384, 200, 131], [60, 1, 2, 3, 4, 5, 6, 300], None, 7, 8, 1, 64, 16, "random"),  # some outside; an empty group
    ([0, 3], [0], [5, 200, 0], None, 2, 4, 2, 64, 16, "run"),                      # an empty prefix
    ([0, 40], [1500], [7] * 40, None, 1, 8, 8, 128, 64, "run"),                    # every head its own keys: 40 rows
    ([0, 3], [200], [0, 30, 200], None, 128, 4, 1, 96, 64, "random"),              # long runs: 1536 rows
]


@pytest.mark.parametrize("case", PREFIX, ids=lambda c: "-".join(str(x) for x in c[4:]) + f"-{len(c[2])}x{c[1][0]}")
def test_prefix_attention(case):
    starts, prefixes, own, news, n, h, hk, d, page, kind = case
    rng = np.random.default_rng(21)
    b = len(own)
    base = [0] * b
    for g, p in enumerate(prefixes):
        for s in range(starts[g], starts[g + 1]):
            base[s] = p
    lengths = [x + y for x, y in zip(base, own)]
    counts = [n] * b if news is None else news
    cache, table = _shared_cache(rng, starts, prefixes, lengths, counts, hk, d, page)
    q = _bf16(rng.standard_normal((b, n, h, d)) * 1.5).transpose(1, 2)  # token by token, as a projection leaves them
    sees, mask = _mask(rng, b, n, kind)
    whole = starts == [0, b]
    for dtype in (torch.float32, torch.bfloat16):
        got = wise.prefix_attention(q, cache, _i32(prefixes), group_starts=None if whole and dtype == torch.float32 else _i32(starts),
                                    new_len=_i32(news), tree_mask=mask, out_dtype=dtype)
        wise.check_device()
        _check(q, cache, table, sees, lengths, counts, got, dtype)
    again = wise.prefix_attention(q, cache, _i32(prefixes), group_starts=_i32(starts), new_len=_i32(news), tree_mask=mask)
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


def test_what_is_not_shared_has_the_bits_of_tree_attention():
    """No whole tile, a group of one, sequences shorter than the prefix."""
    rng = np.random.default_rng(22)
    lengths = [100, 70, 300, 290]
    cache, table = _shared_cache(rng, [0, 0], [0], lengths, [3] * 4, 2, 128, 32)
    q = _bf16(rng.standard_normal((4, 8, 3, 128)))
    want = wise.tree_attention(q, cache)
    for starts, prefix in (([0, 2], [64]), ([0, 4], [127]), ([2, 3], [256]), ([0, 3], [256]), ([4, 4], [300]), ([0, 4], [400])):
        got = wise.prefix_attention(q, cache, _i32(prefix), group_starts=_i32(starts))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (starts, prefix)
        # (the last prefix is longer than the page table, 11 pages of 32, holds)
        assert wise.device_status() == (wise._lib.WISE_ERR_BAD_CACHE if prefix[0] > table.shape[1] * 32 else 0)


def test_padded_batch():
    """Empty places of a padded batch, the first of a group among them, share
    nothing and hold nothing."""
    rng = np.random.default_rng(23)
    starts, prefixes, lengths, news = [0, 5], [400], [0, 410, 0, 400, 455], [0, 2, 0, 1, 2]
    cache, table = _shared_cache(rng, starts, prefixes, lengths, news, 2, 64, 16)
    q = _bf16(rng.standard_normal((5, 4, 2, 64)))
    for s in range(5):
        q[s, :, news[s]:] = float("nan")
    got = wise.prefix_attention(q, cache, _i32(prefixes), group_starts=_i32(starts), new_len=_i32(news), out_dtype=torch.float32)
    wise.check_device()
    q = torch.nan_to_num(q)
    sees = _mask(rng, 5, 2, "run")[0]
    _check(q, cache, table, sees, lengths, news, got, torch.float32)


@pytest.mark.parametrize("d,h,n,members", [(128, 32, 1, 64), (64, 8, 2, 8), (96, 40, 5, 24)])
def test_long_prefixes_equal_the_attention_without_sharing(d, h, n, members):
    """Units cut over many blocks, rings gone round: against tree_attention of
    the same cache, each within its bound of the exact values."""
    g = torch.Generator(device="cuda").manual_seed(5)
    hk, page, prefix = 8 if h > 8 else 2, 64, 16411
    whole, own = prefix // page, 5
    table = torch.full((members, whole + own + 1), -1, dtype=torch.int32, device="cuda")
    order = torch.randperm(whole + own * members, generator=g, device="cuda").to(torch.int32)
    table[:, :whole] = order[:whole]
    table[:, whole:whole + own] = order[whole:].reshape(members, own)
    k, v = (torch.randn((order.numel(), hk, page, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    left = prefix % page
    for p in (k, v):
        p[table[1:, whole].long(), :, :left] = p[int(table[0, whole]), :, :left]
    lengths = prefix + torch.randint(0, own * page - left - n, (members,), generator=g, device="cuda").to(torch.int32)
    cache = wise.PagedCache(k, v, table, lengths.to(torch.int32))
    q = torch.randn((members, h, n, d), generator=g, device="cuda").to(torch.bfloat16)
    pre = torch.tensor([prefix], dtype=torch.int32, device="cuda")
    o, lse = wise.prefix_attention(q, cache, pre, out_dtype=torch.float32)
    ro, rl = wise.tree_attention(q, cache, out_dtype=torch.float32)
    wise.check_device()
    # sum a |v| of a row is below 1.2 here (16K values, E |v| = 0.8, weights in nobody's favour); each side's
    # O is off by at most (2 * 2^-8 + 2^-10) of it, with scores of size up to 64: e_s < 2^-12
    assert float((o - ro).abs().max()) <= 2 * (2.0 ** -7 + 2.0 ** -10) * 1.2
    assert float((lse - rl).abs().max()) <= 2 * (2.0 ** -12 + 2.0 ** -20 + 2.0 ** -24 * (64 + prefix / 8 + 40))


def test_non_finite_values_of_new_tokens_reach_only_rows_that_see_them():
    rng = np.random.default_rng(24)
    starts, prefixes, lengths = [0, 3], [256], [300, 256, 270]
    cache, table = _shared_cache(rng, starts, prefixes, lengths, [4] * 3, 2, 64, 16)
    q = _bf16(rng.standard_normal((3, 4, 4, 64)))
    pg, row = C.slot(table, 1, 256 + 2, 16)  # new token 2 of sequence 1
    want = wise.prefix_attention(q, cache, _i32(prefixes), out_dtype=torch.float32)[0]
    cache.v_pages[pg, :, row, 5] = float("inf")
    got = wise.prefix_attention(q, cache, _i32(prefixes), out_dtype=torch.float32)[0]
    hit = torch.zeros_like(want, dtype=torch.bool)
    hit[1, :, 2:, 5] = True
    assert torch.all(torch.isinf(got[hit])) and torch.equal(got[~hit], want[~hit])


def test_bad_entries_are_flagged():
    rng = np.random.default_rng(25)
    lengths = [300, 280, 290]
    cache, table = _shared_cache(rng, [0, 3], [256], lengths, [1] * 3, 2, 64, 32)
    q = _bf16(rng.standard_normal((3, 4, 1, 64)))
    want = wise.tree_attention(q, cache)
    wise.check_device()
    # starts that do not ascend, or leave the batch: nothing is shared
    for starts, prefix in (([0, 3, 1], [256, 256]), ([-1, 3], [256]), ([0, 4], [256]), ([0, 2, 1, 3], [256, 128, 256])):
        got = wise.prefix_attention(q, cache, _i32(prefix), group_starts=_i32(starts))
        with pytest.raises(wise.WiseError):
            wise.check_device()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # prefixes out of range: negative ones share nothing, ones past the table are longer than every sequence
    for prefix in (-5, 1 << 30):
        got = wise.prefix_attention(q, cache, _i32([prefix]))
        with pytest.raises(wise.WiseError):
            wise.check_device()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # a shared page outside the pool is not seen by anyone
    bad = table.copy()
    bad[:, 3] = cache.k_pages.shape[0]
    broken = wise.PagedCache(cache.k_pages, cache.v_pages, _i32(bad), cache.lengths)
    o, lse = wise.prefix_attention(q, broken, _i32([256]), out_dtype=torch.float32)
    with pytest.raises(wise.WiseError):
        wise.check_device()
    ro, rl = wise.tree_attention(q, broken, out_dtype=torch.float32)
    with pytest.raises(wise.WiseError):
        wise.check_device()
    assert torch.all(torch.isfinite(o)) and float((lse - rl).abs().max()) <= 2.0 ** -16
    assert float((o - ro).abs().max()) <= 2 * (2.0 ** -7 + 2.0 ** -10) * 4.0  # |v| < 4


def test_a_shared_batch_from_prompt_to_eviction():
    """One prompt in shared pages, four samples behind it: appended with norms,
    attended to as a shared batch, weighed, cut down to pages of their own."""
    g = torch.Generator(device="cuda").manual_seed(9)
    b, h, hk, d, page, prompt, budget = 4, 8, 2, 64, 32, 288, 96
    shared = prompt // page
    k, v = (torch.zeros((shared + 4 * b + 3 * b, hk, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rope, kn, qn = wise.rope_frequencies(d), torch.rand(d, generator=g, device="cuda") + 0.5, torch.rand(d, generator=g, device="cuda") + 0.5
    table = torch.full((b, shared + 4), -1, dtype=torch.int32, device="cuda")
    table[:, :shared] = torch.arange(shared, device="cuda")
    table[:, shared:] = shared + torch.arange(4 * b, device="cuda").reshape(b, 4)

    def draw(batch, m, n):
        return torch.randn((batch, m, n, d), generator=g, device="cuda").to(torch.bfloat16)
    first = wise.PagedCache(k, v, table[:1].contiguous(), _i32([0]))
    x = draw(1, hk, prompt), draw(1, hk, prompt)
    wise.cache_append(first, *x, rope=rope, k_norm=kn)
    cache = wise.PagedCache(k, v, table, _i32([prompt] * b))
    weights = torch.zeros((b, hk, 400), device="cuda")
    pre = _i32([prompt])
    for step in range(5):
        qkv = draw(b, h, 1), draw(b, hk, 1), draw(b, hk, 1)
        q = wise.cache_append(cache, qkv[1], qkv[2], q=qkv[0], rope=rope, q_norm=qn, k_norm=kn)
        o, lse = wise.prefix_attention(q, cache, pre, out_dtype=torch.float32)
        ro, rl = wise.tree_attention(q, cache, out_dtype=torch.float32)
        assert float((lse - rl).abs().max()) <= 2.0 ** -16 and float((o - ro).abs().max()) <= 2 * (2.0 ** -7 + 2.0 ** -10) * 4.0
        wise.cache_weights(q, cache, lse, weights)
        cache.lengths = wise.cache_accept(cache, _i32([1] * b))
    assert torch.all((weights[:, :, :prompt + 5].sum(-1) - 5 * h // hk).abs() < 5 * h // hk * 2.0 ** -12)
    to = (shared + 4 * b + torch.arange(3 * b, device="cuda").reshape(b, 3)).to(torch.int32)
    small, kept = wise.cache_evict(cache, weights, budget, to.contiguous(), recent=5, sink=2)
    wise.check_device()
    wn = weights.cpu().numpy()
    for s in range(b):
        for y in range(hk):
            for i, t in enumerate(C.kept_tokens(wn[s, y], prompt + 5, budget, 5, 2)):
                a, c = C.slot(table.tolist(), s, t, page), C.slot(to.tolist(), s, i, page)
                assert torch.equal(k[a[0], y, a[1]], k[c[0], y, c[1]]) and torch.equal(v[a[0], y, a[1]], v[c[0], y, c[1]])
                assert float(kept[s, y, i]) == float(wn[s, y, t])
