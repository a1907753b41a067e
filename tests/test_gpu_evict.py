"""Attention weight gathered by cached tokens, and eviction by it, on the GPU
against the formulas in 64 bits.

Tolerance of the weights. A score is exact products summed in fp32, off by
(d + 8) 2^-24 of the sum of their sizes; the exponent's product, the LSE in
powers of two and their difference round by 2^-22 of |score| + |LSE|; the
exponential is off by 2^-22. With e the sum of sizes plus |LSE| plus 1, a row's
weight p is off by less than (d + 16) 2^-24 p e. R of them are summed in R + 4
roundings of 2^-24 of the whole.
An eviction moves values: equal bits.
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


def _table(rng, totals, page, spare_pages=2):
    used = [(t + page - 1) // page for t in totals]
    order = rng.permutation(sum(used) + spare_pages)
    table = np.full((len(totals), max(max(used), 1) + 1), -1, np.int32)
    at = 0
    for s, u in enumerate(used):
        table[s, :u] = order[at:at + u]
        at += u
    return table, sum(used) + spare_pages, [int(x) for x in order[at:]]


def _pool(rng, hk, d, page, table, n_pages, totals):
    """Random values in every token's row, NaN elsewhere."""
    k = np.full((n_pages, hk, page, d), np.nan, np.float32)
    for s, total in enumerate(totals):
        for t in range(total):
            pg, row = C.slot(table, s, t, page)
            k[pg, :, row] = rng.standard_normal((hk, d))
    return _bf16(k)


def _sees(rng, b, n, kind):
    if kind == "random":
        m = rng.random((b, n, n)) < 0.4
        m[:, n // 2] = False
        return m
    return np.broadcast_to(np.tril(np.ones((n, n), bool)), (b, n, n)).copy()


# (lengths, new_len, n, heads, kv_heads, d, page, mask)
WEIGHTS = [
    ([5], None, 1, 2, 2, 64, 16, "run"),
    ([0], None, 1, 1, 1, 128, 16, "run"),
    ([127, 128, 129], None, 1, 8, 2, 128, 64, "run"),
    ([1, 130, 0, 16], [7, 3, 5, 0], 7, 8, 2, 64, 16, "random"),
    ([250, 3], [13, 9], 13, 5, 5, 96, 32, "run"),
    ([300], None, 16, 16, 1, 128, 128, "random"),       # 256 rows
    ([140, 40], [33, 17], 33, 10, 1, 96, 32, "random"),  # 330 rows: two launches
    ([60], [70], 128, 8, 1, 64, 64, "run"),             # 1024 rows, four launches, the last without a token
    ([520, 3, 90], None, 5, 4, 2, 128, 16, "random"),
]


@pytest.mark.parametrize("case", WEIGHTS, ids=lambda c: "-".join(str(x) for x in c[2:]))
def test_weights(case):
    lengths, news, n, h, hk, d, page, kind = case
    rng = np.random.default_rng(2)
    b = len(lengths)
    totals = [x + (n if news is None else news[s]) for s, x in enumerate(lengths)]
    table, n_pages, _ = _table(rng, totals, page)
    cache = wise.PagedCache(_pool(rng, hk, d, page, table, n_pages, totals), _pool(rng, hk, d, page, table, n_pages, totals),
                            _i32(table), _i32(lengths))
    q = _bf16(rng.standard_normal((b, h, n, d)) * 1.3)
    sees = _sees(rng, b, n, kind)
    mask = wise.pack_tree_mask(torch.from_numpy(sees).cuda()) if kind == "random" else None
    _, lse = wise.tree_attention(q, cache, new_len=_i32(news), tree_mask=mask)
    for s in range(b):  # what padding rows hold has no influence
        if news is not None:
            q[s, :, news[s]:] = float("nan")
    lse[:, 0, 0] = -float("inf")  # a row that the caller leaves out
    width = max(totals) + 3
    start = rng.random((b, hk, width)).astype(np.float32)
    for s in range(b):
        start[s, :, lengths[s]:totals[s]] = np.nan  # new tokens' entries are written
    weights = torch.from_numpy(start).cuda()
    got = wise.cache_weights(q, cache, lse, weights, new_len=_i32(news), tree_mask=mask)
    wise.check_device()
    assert got is weights
    qn = _np(q)
    want, size = C.gather_weights(np.nan_to_num(qn), _np(cache.k_pages), table, lengths, sees, _np(lse), start.astype(np.float64),
                                  news)
    rows = h // hk * n
    tol = (d + 16) * 2.0 ** -24 * size + (rows + 4) * 2.0 ** -24 * np.abs(want)
    off = np.abs(_np(got) - want)
    assert np.all(off <= tol), f"{np.nanmax(off - tol):.3e} past the bound"
    changed = size > 0
    assert np.array_equal(_np(got)[~changed & ~np.isnan(start)], want[~changed & ~np.isnan(start)])
    # the same bits again
    again = torch.from_numpy(start).cuda()
    wise.cache_weights(q, cache, lse, again, new_len=_i32(news), tree_mask=mask)
    assert torch.equal(again, got)


def test_weights_of_long_sequences_sum_to_the_rows():
    """Each row's weights sum to 1: over many tiles, sequences and rings."""
    rng = np.random.default_rng(4)
    lengths, n, h, hk, d, page = [40000, 17, 9000, 0, 25000], 3, 8, 2, 64, 64
    table, n_pages, _ = _table(rng, [x + n for x in lengths], page)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((n_pages, hk, page, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    cache = wise.PagedCache(k, v, _i32(table), _i32(lengths))
    q = torch.randn((5, h, n, d), generator=g, device="cuda").to(torch.bfloat16)
    _, lse = wise.tree_attention(q, cache)
    weights = torch.zeros((5, hk, max(lengths) + n), device="cuda")
    wise.cache_weights(q, cache, lse, weights)
    wise.check_device()
    total = weights.double().sum(-1)
    # LSE is off by the bound of its own tests, some 2^-10 here
    assert torch.all((total - h // hk * n).abs() <= h // hk * n * 2.0 ** -10)


# (lengths, budget, recent, sink, kv_heads, d, page, spread)
EVICT = [
    ([10], 4, 1, 1, 1, 64, 16, "plain"),
    ([0, 1, 5, 6, 7], 5, 2, 1, 2, 64, 16, "plain"),
    ([300, 40, 299], 64, 0, 0, 3, 96, 32, "ties"),
    ([1000], 1000, 10, 10, 2, 128, 64, "plain"),       # nothing to evict
    ([1000, 2000], 999, 999, 0, 2, 128, 64, "plain"),  # recent ones only
    ([500], 20, 0, 20, 2, 64, 128, "plain"),           # sinks only
    ([700, 650], 333, 33, 4, 2, 96, 16, "equal"),      # every weight the same
    ([700], 333, 33, 4, 2, 64, 16, "odd"),             # infinities, NaN, zeros of both signs, negative
    ([3000, 1, 2999], 1, 0, 0, 1, 64, 16, "plain"),
]


def _spread(rng, shape, kind):
    w = np.exp(3 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        w = np.round(w)
    elif kind == "equal":
        w[:] = 0.25
    elif kind == "odd":
        pick = rng.integers(0, 8, shape)
        for i, x in enumerate((np.inf, -np.inf, np.nan, 0.0, -0.0, -1.5, 1e-42)):
            w[pick == i] = x
    return w


@pytest.mark.parametrize("case", EVICT, ids=lambda c: "-".join(str(x) for x in c[1:]))
def test_evict(case):
    lengths, budget, recent, sink, hk, d, page, kind = case
    _run_evict(np.random.default_rng(6), lengths, budget, recent, sink, hk, d, page, kind, max(lengths) + 2, None)


def _run_evict(rng, lengths, budget, recent, sink, hk, d, page, kind, width, width_out, extra_cols=0):
    b = len(lengths)
    kept = [min(x, budget) for x in lengths]
    need = sum((x + page - 1) // page for x in kept)
    table, n_pages, free = _table(rng, lengths, page, need + 2)
    if extra_cols:  # a page table for far longer sequences
        table = np.concatenate([table, np.full((b, extra_cols), -1, np.int32)], 1)
    to = np.full((b, (budget + page - 1) // page + 1), -1, np.int32)
    for s, x in enumerate(kept):
        for c in range((x + page - 1) // page):
            # a sequence that keeps everything may stay where it is
            to[s, c] = table[s, c] if lengths[s] <= budget and s % 2 else free.pop()
    # every row of the pools is told apart by its first values
    pools = []
    for x in range(2):
        p = np.arange(n_pages * hk * page).reshape(n_pages, hk, page, 1)
        p = np.concatenate([p % 251, p // 251 % 251, p // 63001, np.full_like(p, x)] + [p % 7] * (d - 4), 3)
        pools.append(_bf16(p))
    before = [_np(p) for p in pools]
    weights = _spread(rng, (b, hk, width), kind)
    cache = wise.PagedCache(pools[0], pools[1], _i32(table), _i32(lengths))
    out = None if width_out is None else torch.full((b, hk, width_out), 9.0, device="cuda")
    new, w = wise.cache_evict(cache, torch.from_numpy(weights).cuda(), budget, _i32(to), recent=recent, sink=sink, weights_out=out)
    wise.check_device()
    kp, vp, want_lengths, want = C.evict(before[0], before[1], table, lengths, weights, budget, to, recent, sink, w.shape[2])
    assert new.lengths.tolist() == want_lengths and new.page_table.tolist() == to.tolist()
    assert np.array_equal(w.cpu().numpy(), want, equal_nan=True)
    assert np.array_equal(_np(new.k_pages), kp) and np.array_equal(_np(new.v_pages), vp)
    assert cache.lengths.tolist() == list(lengths)


@pytest.mark.parametrize("kind", ["plain", "ties", "equal"])
def test_evict_from_long_sequences_by_clusters(kind):
    """Page tables of more than 16K tokens: eight blocks share a key head; past
    128K they read the weights again."""
    _run_evict(np.random.default_rng(8), [20000, 33, 18001], 1500, 100, 4, 2, 64, 64, kind, 20011, 1600)
    _run_evict(np.random.default_rng(9), [140001], 2000, 0, 3, 1, 64, 128, kind, 140001, 2000)


def test_evict_many_heads_of_long_tables_by_single_blocks():
    _run_evict(np.random.default_rng(10), [17000, 300], 500, 20, 4, 160, 64, 128, "ties", 17000, 500)
    # short sequences behind a table of 16K and more
    _run_evict(np.random.default_rng(12), [100, 5000], 90, 10, 4, 3, 64, 16, "ties", 5000, 96, extra_cols=1100)


def test_evicted_cache_attends_and_grows():
    """A cache cut down by its own weights: attention over what is kept equals
    attention with the others left out, and the cache goes on from there."""
    rng = np.random.default_rng(13)
    lengths, n, h, hk, d, page, budget = [180, 60], 2, 4, 2, 64, 16, 70
    table, n_pages, free = _table(rng, [x + 8 for x in lengths], page, 30)
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn((n_pages, hk, page, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    cache = wise.PagedCache(k, v, _i32(table), _i32(lengths))
    rope = wise.rope_frequencies(d)
    x = [torch.randn((2, m, n, d), generator=g, device="cuda").to(torch.bfloat16) for m in (hk, hk, h)]
    q = wise.cache_append(cache, x[0], x[1], q=x[2], rope=rope)
    _, lse = wise.tree_attention(q, cache)
    weights = torch.zeros((2, hk, 200), device="cuda")
    wise.cache_weights(q, cache, lse, weights)
    cache.lengths = wise.cache_accept(cache, _i32([n, n]))
    to = _i32([[free.pop() for _ in range(6)] for _ in range(2)])
    small, kept = wise.cache_evict(cache, weights, budget, to, recent=8, sink=2)
    wise.check_device()
    assert small.lengths.tolist() == [70, 62]
    new = [torch.randn((2, m, 1, d), generator=g, device="cuda").to(torch.bfloat16) for m in (hk, hk, h)]
    at = cache.lengths[:, None].contiguous()  # the next token's position, whatever its slot
    qr = wise.cache_append(small, new[0], new[1], q=new[2], positions=at, rope=rope)
    o, lse = wise.tree_attention(qr, small, out_dtype=torch.float32)
    grown = wise.cache_weights(qr, small, lse, kept)
    wise.check_device()
    wn = weights.cpu().numpy()
    for s in range(2):
        for y in range(hk):
            keep = C.kept_tokens(wn[s, y], lengths[s] + n, budget, 8, 2)
            rows = [C.slot(table, s, t, page) for t in keep]
            last = C.slot(to.tolist(), s, len(keep), page)
            ks = torch.stack([cache.k_pages[p, y, r] for p, r in rows + [last]]).double()
            vs = torch.stack([cache.v_pages[p, y, r] for p, r in rows] + [new[1][s, y, 0]]).double()
            for z in range(y * 2, y * 2 + 2):
                p = torch.softmax(qr[s, z, 0].double() @ ks.T / 8.0, -1)
                # the weights' rounding (2 * 2^-8, as in the attention's tests), and its exponent's
                tol = (2.0 ** -7 + 2.0 ** -12) * (p[:, None] * vs.abs()).sum(0)
                assert torch.all((o[s, z, 0].double() - p @ vs).abs() <= tol)
            assert torch.all(grown[s, y, :len(keep) + 1] > 0) and torch.all(grown[s, y, len(keep) + 1:] == 0)


def test_bad_entries_are_flagged_and_skipped():
    rng = np.random.default_rng(14)
    table, n_pages, free = _table(rng, [60], 16, 6)
    k = _pool(rng, 1, 64, 16, table, n_pages, [60])
    weights = torch.from_numpy(rng.random((1, 1, 64)).astype(np.float32)).cuda()
    weights[..., 16:32] += 1.0  # the second page's tokens are always among the kept
    good = wise.PagedCache(k, k.clone(), _i32(table), _i32([59]))
    q = _bf16(rng.standard_normal((1, 2, 1, 64)))
    _, lse = wise.tree_attention(q, good)
    for what in ("page", "length", "width"):
        t2, l2, w2 = table.copy(), [59], weights.clone()
        if what == "page":
            t2[0, 1] = n_pages
        elif what == "length":
            l2 = [200]  # past the table
        else:
            w2 = w2[:, :, :40].contiguous()
        cache = wise.PagedCache(k, k.clone(), _i32(t2), _i32(l2))
        start = w2.clone()
        wise.cache_weights(q, cache, lse, w2)
        with pytest.raises(wise.WiseError):
            wise.check_device()
        if what == "page":  # its tokens gather nothing, the others as ever
            ref = weights.clone()
            wise.cache_weights(q, good, lse, ref)
            assert torch.equal(w2[..., 16:32], start[..., 16:32])
            assert torch.equal(w2[..., :16], ref[..., :16]) and torch.equal(w2[..., 32:], ref[..., 32:])
        to = _i32([[free[0], free[1]]])
        cache.lengths = _i32(l2 if what != "width" else [59])
        before = cache.k_pages.clone()
        new, kept = wise.cache_evict(cache, w2.contiguous(), 20, to, recent=2)
        with pytest.raises(wise.WiseError):
            wise.check_device()
        assert new.lengths.tolist() == [20]
        rest = [p for p in range(n_pages) if p not in (free[0], free[1])]
        assert torch.equal(torch.nan_to_num(cache.k_pages[rest]), torch.nan_to_num(before[rest]))
    wise.check_device()
    # a new page outside the pool
    new, kept = wise.cache_evict(good, weights, 20, _i32([[free[0], n_pages]]))
    with pytest.raises(wise.WiseError):
        wise.check_device()
    assert new.lengths.tolist() == [20]
