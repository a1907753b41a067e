"""The paged-cache operators on the GPU against the fp64 oracle.

Tolerances. A rounding to bf16 is off by at most 2^-8 of the value, one in
fp32 by 2^-24.
 * append: one rounding to bf16 of a rotation taken in fp32. The angle is
   reduced in whole numbers; its top 32 bits as fp32 (2^-23), the sine and
   cosine (2^-21.1 on [-pi, pi]) and the two products and their sum (2^-23)
   are off by less than 2^-20 of |x| + |y|.
 * attention: the scores are exact products summed in fp32, off by at most
   e_s = (d + 8) 2^-24 * scale * sum |q k|, plus 2^-22 for the exponential;
   a weight is rounded to bf16 (2^-8), in the numerator and in the sum that
   divides it alike, so O is off by at most (2 * 2^-8 + 2 e_s + 2^-20) *
   sum a |v|, plus the output's own rounding.
 * LSE: e_s, plus 2^-20 for the exponentials and the logarithm, plus 2^-24
   for every addition of the longest chain of the sum and of its value.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import block_sparse_attention_causal_gb300 as wise
from block_sparse_attention_causal_gb300 import _lib
from oracle import cache_oracle as C
from oracle import wise_oracle as O

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

BF16, F32 = 2.0 ** -8, 2.0 ** -24


def _bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _table(rng, totals, page, spare_cols=1, spare_pages=2):
    """A page table that hands every sequence its own random pages; entries
    past its last token are -1."""
    used = [(t + page - 1) // page for t in totals]
    n_pages = sum(used) + spare_pages
    order = rng.permutation(n_pages)
    table = np.full((len(totals), max(used) + spare_cols), -1, np.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    return table, n_pages


def _pools(rng, hk, d, page, table, n_pages, totals, fill=np.nan, scale=1.0):
    """Pools that hold random values in every token's row and `fill` (NaN)
    everywhere else: no result may depend on what lies there."""
    k = np.full((n_pages, hk, page, d), fill, np.float32)
    v = np.full((n_pages, hk, page, d), fill, np.float32)
    for b, total in enumerate(totals):
        for t in range(total):
            pg, row = C.slot(table, b, t, page)
            k[pg, :, row] = rng.standard_normal((hk, d)) * scale
            v[pg, :, row] = rng.standard_normal((hk, d))
    return _bf16(k), _bf16(v)


def _cache(k, v, table, lengths):
    return wise.PagedCache(k.cuda(), v.cuda(), torch.from_numpy(np.asarray(table, np.int32)).cuda(),
                           torch.tensor(list(lengths), dtype=torch.int32).cuda())


def _i32(x):
    return None if x is None else torch.tensor(np.asarray(x).tolist(), dtype=torch.int32).cuda()


def _tree(rng, b, n, kind):
    """Who sees whom among drafted tokens."""
    if kind == "run":
        return np.broadcast_to(np.tril(np.ones((n, n), bool)), (b, n, n)).copy()
    if kind == "random":  # any bits: rows that see nothing new, tokens that see later ones
        m = rng.random((b, n, n)) < 0.4
        m[:, n // 2] = False
        return m
    m = np.zeros((b, n, n), bool)
    for s in range(b):
        for i in range(n):
            p = int(rng.integers(-1, i)) if i else -1
            if p >= 0:
                m[s, i] = m[s, p]
            m[s, i, i] = True
    return m


def _check_attention(q, cache, sees, lengths, news, table, *, dtype=torch.float32, mask=None, scale=0.0, **kw):
    d, n = q.shape[3], q.shape[2]
    o, lse = wise.tree_attention(q, cache, new_len=_i32(news), tree_mask=mask, out_dtype=dtype, scale=scale, **kw)
    wise.check_device()
    kp, vp = _np(cache.k_pages), _np(cache.v_pages)
    want, want_lse, weight, size = C.tree_attention(_np(q), kp, vp, table, lengths, sees, news, scale or None)
    got, got_lse = _np(o), _np(lse)
    e_s = (d + 8) * F32 * size[..., None]
    tol = (2 * BF16 + 2 * e_s + 2.0 ** -20) * weight + (BF16 * np.abs(want) if dtype == torch.bfloat16 else 0.0)
    assert np.all(np.isfinite(got))
    off = np.abs(got - want)
    assert np.all(off <= tol), f"O: {np.max(off - tol):.3e} past the bound"
    empty = np.isneginf(want_lse)
    assert np.all(got[empty] == 0) and np.all(np.isneginf(got_lse[empty]))
    keys = max(x + y for x, y in zip(lengths, [n] * len(lengths) if news is None else news))
    lse_tol = e_s[..., 0] + 2.0 ** -20 + F32 * (64 + keys / 8 + 2 * np.abs(np.where(empty, 0, want_lse)))
    off = np.abs(got_lse[~empty] - want_lse[~empty])
    assert np.all(off <= lse_tol[~empty]), f"LSE: {np.max(off - lse_tol[~empty]):.3e} past the bound"
    return o, lse


# (batch lengths, new_len, n, heads, kv_heads, d, page, mask)
ATTEND = [
    ([5], None, 1, 2, 2, 64, 16, "run"),                       # a next token behind a few
    ([0], None, 1, 1, 1, 128, 16, "run"),                      # the very first token
    ([0, 0], [1, 0], 3, 4, 2, 96, 32, "tree"),                 # nothing at all in one sequence
    ([127, 128, 129], None, 1, 8, 2, 128, 64, "run"),          # around a tile of 128
    ([1, 130, 0, 16], [7, 3, 5, 0], 7, 8, 2, 64, 16, "tree"),
    ([250, 3], [13, 9], 13, 5, 5, 96, 32, "tree"),             # every head its own keys
    ([120], None, 16, 16, 1, 128, 128, "random"),              # one key head, 256 rows
    ([300, 77], [33, 64], 64, 8, 2, 128, 64, "tree"),
    ([100, 255], [128, 1], 128, 8, 1, 64, 32, "random"),       # 1024 rows
    ([1000, 31, 512], [40, 2, 17], 40, 6, 2, 96, 16, "tree"),
    ([2047, 1], None, 2, 4, 4, 128, 128, "run"),
    ([383], None, 128, 3, 1, 128, 16, "run"),                  # drafted tokens over two tiles
]


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "len%s_n%d_h%d_%d_d%d_p%d_%s" % (
    "-".join(map(str, c[0])), c[2], c[3], c[4], c[5], c[6], c[7]))
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_attention(case, dtype):
    lengths, news, n, h, hk, d, page, kind = case
    rng = np.random.default_rng(sum(lengths) + n + d)
    b = len(lengths)
    totals = [x + y for x, y in zip(lengths, news or [n] * b)]
    table, n_pages = _table(rng, [max(t, 1) for t in totals], page)
    k, v = _pools(rng, hk, d, page, table, n_pages, totals)
    cache = _cache(k, v, table, lengths)
    q = _bf16(rng.standard_normal((b, h, n, d)) * 1.5).cuda()
    sees = _tree(rng, b, n, kind)
    mask = None if kind == "run" else wise.pack_tree_mask(torch.from_numpy(sees).cuda())
    _check_attention(q, cache, sees, lengths, news, table, dtype=dtype, mask=mask)


@pytest.mark.parametrize("heads", [(32, 8), (8, 8), (12, 1)])
def test_attention_of_a_long_cache(heads):
    """Rows split over many blocks and joined again, lengths that differ."""
    h, hk = heads
    rng = np.random.default_rng(h)
    lengths, page, d, n = [5000, 17, 2200], 64, 128, 1
    totals = [x + n for x in lengths]
    table, n_pages = _table(rng, totals, page)
    k, v = _pools(rng, hk, d, page, table, n_pages, totals)
    cache = _cache(k, v, table, lengths)
    q = _bf16(rng.standard_normal((3, h, n, d)) * 2).cuda()
    sees = _tree(rng, 3, n, "run")
    a = _check_attention(q, cache, sees, lengths, None, table)
    b = _check_attention(q, cache, sees, lengths, None, table)
    assert all(torch.equal(x, y) for x, y in zip(a, b))  # joined in a fixed order


@pytest.mark.parametrize("shape", [(64, 16, 4, 1, 1), (96, 32, 4, 4, 1), (128, 64, 8, 2, 1), (128, 128, 2, 1, 50),
                                   (128, 16, 4, 1, 41), (96, 64, 3, 1, 90)], ids=lambda s: "d%d_p%d_h%d_%d_n%d" % s)
def test_long_parts_of_the_line(shape):
    """Every block works through more key tiles than its ring of slots holds,
    over several sequences: 40 sequences, of which three are checked."""
    d, page, h, hk, n = shape
    rng = np.random.default_rng(d + n)
    b, check = 40, [0, 17, 39]
    lengths = [int(x) for x in rng.integers(2000, 6000, b)]
    totals = [x + n for x in lengths]
    table, n_pages = _table(rng, totals, page)
    g = torch.Generator(device="cuda").manual_seed(d)
    k, v = (torch.randn((n_pages, hk, page, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    cache = wise.PagedCache(k, v, _i32(table), _i32(lengths))
    q = _bf16(rng.standard_normal((b, h, n, d)) * 1.5).cuda()
    rows = [n - 1] if n == 1 else [0, n // 2, n - 1]  # rows of the checked sequences
    o, lse = wise.tree_attention(q, cache, out_dtype=torch.float32)
    wise.check_device()
    for s in check:
        pages = torch.from_numpy(table[s][:(totals[s] + page - 1) // page].astype(np.int64)).cuda()
        kk, vv = (x[pages].transpose(0, 1).reshape(hk, -1, d)[:, :totals[s]].double().cpu().numpy() for x in (k, v))
        for y in range(h):
            for i in rows:
                m = lengths[s] + i + 1
                x = y // (h // hk)
                qi = _np(q)[s, y, i]
                sc = kk[x, :m] @ qi / np.sqrt(d)
                p = np.exp(sc - sc.max())
                want, weight = p @ vv[x, :m] / p.sum(), p @ np.abs(vv[x, :m]) / p.sum()
                e_s = (d + 8) * F32 * (np.abs(kk[x, :m]) @ np.abs(qi)).max() / np.sqrt(d)
                assert np.all(np.abs(_np(o)[s, y, i] - want) <= (2 * BF16 + 2 * e_s + 2.0 ** -20) * weight)
                tol = e_s + 2.0 ** -20 + F32 * (64 + m / 8 + 2 * 12)
                assert abs(float(lse[s, y, i]) - (sc.max() + np.log(p.sum()))) <= tol
    again = wise.tree_attention(q, cache, out_dtype=torch.float32)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def test_many_sequences():
    rng = np.random.default_rng(7)
    b, page, d = 700, 16, 64
    lengths = [int(x) for x in rng.integers(0, 40, b)]
    news = [int(x) for x in rng.integers(0, 3, b)]
    totals = [x + y for x, y in zip(lengths, news)]
    table, n_pages = _table(rng, [max(t, 1) for t in totals], page)
    k, v = _pools(rng, 1, d, page, table, n_pages, totals)
    cache = _cache(k, v, table, lengths)
    q = _bf16(rng.standard_normal((b, 2, 2, d))).cuda()
    _check_attention(q, cache, _tree(rng, b, 2, "run"), lengths, news, table)


def test_peaked_rows_and_large_scores():
    """One key far above the rest, in any tile: the running maximum moves."""
    rng = np.random.default_rng(11)
    lengths, page, d, n = [900], 32, 128, 3
    table, n_pages = _table(rng, [903], page)
    k, v = _pools(rng, 1, d, page, table, n_pages, [903])
    kk = k.float().numpy()
    q = rng.standard_normal((1, 2, n, d))
    for t, x in ((10, 1.0), (140, 3.0), (500, 6.0), (880, 2.0)):
        pg, row = C.slot(table, 0, t, page)
        kk[pg, 0, row] = q[0, 0, 0] * x
    cache = _cache(_bf16(kk), v, table, lengths)
    _check_attention(_bf16(q).cuda(), cache, _tree(rng, 1, n, "run"), lengths, None, table)
    _check_attention(_bf16(q * 20).cuda(), cache, _tree(rng, 1, n, "run"), lengths, None, table)
    _check_attention(_bf16(q).cuda(), cache, _tree(rng, 1, n, "run"), lengths, None, table, scale=0.9)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_unseen_drafted_tokens_have_no_influence(bad):
    """NaN and infinities in the keys and values of drafted tokens reach the
    rows that see them and no others."""
    rng = np.random.default_rng(13)
    lengths, page, d, n = [130, 0], 16, 64, 6
    totals = [x + n for x in lengths]
    table, n_pages = _table(rng, totals, page)
    k, v = _pools(rng, 2, d, page, table, n_pages, totals)
    sees = np.zeros((2, n, n), bool)
    for i in range(n):
        sees[:, i, i] = True
    sees[:, 3, 2] = True  # token 3 sees token 2, which is spoilt; nobody else does
    q = _bf16(rng.standard_normal((2, 4, n, d))).cuda()
    mask = wise.pack_tree_mask(torch.from_numpy(sees).cuda())
    clean = _cache(k, v, table, lengths)
    want, want_lse = _check_attention(q, clean, sees, lengths, None, table, mask=mask)
    for pool in ("v", "k"):
        kk, vv = k.clone(), v.clone()
        for b in range(2):
            pg, row = C.slot(table, b, lengths[b] + 2, page)
            (vv if pool == "v" else kk)[pg, :, row, 5] = bad
        o, lse = wise.tree_attention(q, _cache(kk, vv, table, lengths), tree_mask=mask, out_dtype=torch.float32)
        wise.check_device()
        rest = [0, 1, 4, 5]
        assert torch.equal(o[:, :, rest], want[:, :, rest]) and torch.equal(lse[:, :, rest], want_lse[:, :, rest])
        if pool == "v":
            for i in (2, 3):
                hit = o[:, :, i, 5]
                assert torch.isnan(hit).all() if np.isnan(bad) else (hit == bad).all()
                other = [x for x in range(d) if x != 5]
                assert torch.equal(o[:, :, i, other], want[:, :, i, other])
            assert torch.equal(lse, want_lse)
        elif np.isnan(bad):
            assert torch.isnan(lse[:, :, [2, 3]]).all() and torch.isnan(o[:, :, [2, 3]]).all()


@pytest.mark.parametrize("n,h,hk", [(40, 4, 2), (70, 8, 2), (128, 1, 1), (20, 3, 1)],
                         ids=lambda x: str(x))
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_unseen_drafted_tokens_have_no_influence_on_wide_units(n, h, hk, bad):
    """The same for units of 60 to 280 rows, drafted tokens over two tiles."""
    rng = np.random.default_rng(n)
    lengths, page, d, spoilt = [70, 250], 32, 128, n // 2
    totals = [x + n for x in lengths]
    table, n_pages = _table(rng, totals, page)
    k, v = _pools(rng, hk, d, page, table, n_pages, totals)
    sees = _tree(rng, 2, n, "tree")
    sees[:, :, spoilt] = False
    seen_by = [spoilt, n - 1]
    sees[:, seen_by, spoilt] = True
    mask = wise.pack_tree_mask(torch.from_numpy(sees).cuda())
    q = _bf16(rng.standard_normal((2, h, n, d))).cuda()
    want, want_lse = _check_attention(q, _cache(k, v, table, lengths), sees, lengths, None, table, mask=mask)
    rest = [x for x in range(n) if x not in seen_by]
    for pool in ("v", "k"):
        kk, vv = k.clone(), v.clone()
        for b in range(2):
            pg, row = C.slot(table, b, lengths[b] + spoilt, page)
            (vv if pool == "v" else kk)[pg, :, row, 77] = bad
        o, lse = wise.tree_attention(q, _cache(kk, vv, table, lengths), tree_mask=mask, out_dtype=torch.float32)
        wise.check_device()
        assert torch.equal(o[:, :, rest], want[:, :, rest]) and torch.equal(lse[:, :, rest], want_lse[:, :, rest])
        if pool == "v":
            hit = o[:, :, seen_by, 77]
            assert torch.isnan(hit).all() if np.isnan(bad) else (hit == bad).all()
            other = [x for x in range(d) if x != 77]
            assert torch.equal(o[:, :, seen_by][..., other], want[:, :, seen_by][..., other])
        elif np.isnan(bad):
            assert torch.isnan(lse[:, :, seen_by]).all() and torch.isnan(o[:, :, seen_by]).all()


@pytest.mark.parametrize("n", [1, 9, 20, 40])
def test_nan_in_a_committed_token_reaches_every_row(n):
    rng = np.random.default_rng(n)
    lengths, page, d, h, hk = [300], 64, 64, 8, 2
    table, n_pages = _table(rng, [300 + n], page)
    k, v = _pools(rng, hk, d, page, table, n_pages, [300 + n])
    q = _bf16(rng.standard_normal((1, h, n, d))).cuda()
    clean = wise.tree_attention(q, _cache(k, v, table, lengths))
    pg, row = C.slot(table, 0, 200, page)
    kk, vv = k.clone(), v.clone()
    kk[pg, 1, row, 3] = float("nan")
    o, lse = wise.tree_attention(q, _cache(kk, v, table, lengths))
    assert torch.isnan(o[:, 4:]).all() and torch.isnan(lse[:, 4:]).all()
    assert torch.equal(o[:, :4], clean[0][:, :4]) and torch.equal(lse[:, :4], clean[1][:, :4])
    vv[pg, 0, row, 5] = float("inf")
    o, lse = wise.tree_attention(q, _cache(k, vv, table, lengths))
    wise.check_device()
    assert (o[:, :4, :, 5] == float("inf")).all() and torch.equal(lse, clean[1])
    assert torch.equal(o[:, 4:], clean[0][:, 4:]) and torch.isfinite(o[:, :4, :, :5]).all()


def test_pools_past_32_bits():
    """Pages whose elements lie past 2^32 in their pool."""
    rng = np.random.default_rng(3)
    page, d, hk, n = 128, 128, 2, 5
    n_pages = (1 << 32) // (page * d * hk) + 8  # 8.6 GB a pool
    k, v = (torch.empty((n_pages, hk, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = np.array([[n_pages - 1, n_pages - 3], [n_pages - 5, n_pages - 2]], np.int32)
    lengths = [0, 0]
    cache = wise.PagedCache(k, v, _i32(table), _i32(lengths))
    x = _bf16(rng.standard_normal((2, hk, 200, d))).cuda()
    y = _bf16(rng.standard_normal((2, hk, 200, d))).cuda()
    wise.cache_append(cache, x, y)
    cache.lengths = _i32([195, 195])
    q = _bf16(rng.standard_normal((2, 4, n, d))).cuda()
    o, lse = wise.tree_attention(q, cache, out_dtype=torch.float32)
    # the same tokens in a small pool
    small = np.array([[0, 1], [2, 3]], np.int32)
    pools = [torch.zeros((4, hk, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    near = wise.PagedCache(*pools, _i32(small), _i32([0, 0]))
    wise.cache_append(near, x, y)
    near.lengths = _i32([195, 195])
    want, want_lse = wise.tree_attention(q, near, out_dtype=torch.float32)
    assert torch.equal(o, want) and torch.equal(lse, want_lse)
    path = _i32([[1, 4, -1], [0, 2, 3]])
    for c in (cache, near):
        c.lengths = wise.cache_accept(c, _i32([2, 3]), path)
    wise.check_device()
    for b in range(2):
        for i in range(2):
            assert torch.equal(k[int(table[b, i])], pools[0][2 * b + i]) or i == 1
            assert torch.equal(v[int(table[b, i]), :, :72], pools[1][2 * b + i, :, :72])


def test_strided_queries_and_given_buffers():
    rng = np.random.default_rng(17)
    lengths, page, d, n, h, hk = [70, 9], 32, 96, 5, 6, 3
    totals = [x + n for x in lengths]
    table, n_pages = _table(rng, totals, page)
    k, v = _pools(rng, hk, d, page, table, n_pages, totals)
    cache = _cache(k, v, table, lengths)
    wide = _bf16(rng.standard_normal((2, n, h + 4, d + 8))).cuda()
    q = wide[:, :, 2:2 + h, :d].transpose(1, 2)
    assert not q.is_contiguous()
    out = torch.full((2, h, n, d), 7.0, dtype=torch.float32, device="cuda")
    lse = torch.full((2, h, n), 7.0, dtype=torch.float32, device="cuda")
    o, l2 = _check_attention(q, cache, _tree(rng, 2, n, "run"), lengths, None, table, out=out, lse=lse)
    assert o.data_ptr() == out.data_ptr() and l2.data_ptr() == lse.data_ptr()
    o2, none = wise.tree_attention(q, cache, want_lse=False, out_dtype=torch.float32)
    assert none is None and torch.equal(o2, o)


def test_equals_discover_on_a_run_of_tokens():
    """The last tokens of a prompt, seen through the cache, are what the
    library's causal attention gives for the whole prompt."""
    rng = np.random.default_rng(19)
    b, h, hk, n, d, page = 2, 4, 2, 384, 128, 64
    x = [_bf16(rng.standard_normal((b, y, n, d))).cuda() for y in (h, hk, hk)]
    want, want_lse, _ = wise.discover(*x, 128, want_mass=False, out_dtype=torch.float32)
    table, n_pages = _table(rng, [n] * b, page)
    empty = torch.full((n_pages, hk, page, d), float("nan"), dtype=torch.bfloat16)
    cache = _cache(empty, empty, table, [0] * b)
    wise.cache_append(cache, x[1], x[2])
    last = 100
    cache.lengths = _i32([n - last] * b)
    o, lse = wise.tree_attention(x[0][:, :, n - last:], cache, out_dtype=torch.float32)
    wise.check_device()
    # both sides stay within their own bound of the same exact values
    a = np.abs(_np(x[2])).max()
    assert np.max(np.abs(_np(o) - _np(want[:, :, n - last:]))) <= 4 * BF16 * a
    assert np.max(np.abs(_np(lse) - _np(want_lse[:, :, n - last:]))) <= 2e-5


# ------------------------------------------------------------------- append

APPEND = [  # lengths, new_len, n, heads (0: no q), kv_heads, d, page, rotary, pairs, positions
    ([0], None, 1, 0, 1, 64, 16, 64, False, False),
    ([5, 0, 31], None, 1, 4, 2, 128, 32, 128, False, False),
    ([15, 16, 17], [3, 0, 20], 20, 3, 3, 96, 16, 96, True, True),
    ([100], None, 200, 2, 1, 64, 64, 32, True, False),
    ([7, 300], [130, 129], 130, 8, 2, 128, 128, 64, False, True),
    ([1], None, 33, 5, 5, 96, 32, 48, False, False),
    ([0, 64], None, 64, 0, 4, 128, 64, 0, False, False),
    ([0], None, 17, 1, 1, 96, 16, 16, True, True),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "len%s_n%d_h%d_%d_d%d_p%d_r%d_%s_%s" % (
    "-".join(map(str, c[0])), *c[2:8], "pairs" if c[8] else "halves", "pos" if c[9] else "seq"))
def test_append(case):
    lengths, news, n, h, hk, d, page, rotary, pairs, given = case
    rng = np.random.default_rng(n + d + rotary)
    b = len(lengths)
    totals = [x + y for x, y in zip(lengths, news or [n] * b)]
    table, n_pages = _table(rng, [max(t, 1) for t in totals], page)
    k0, v0 = _bf16(rng.standard_normal((n_pages, hk, page, d))), _bf16(rng.standard_normal((n_pages, hk, page, d)))
    cache = _cache(k0, v0, table, lengths)
    # one projection's output: queries, keys and values of a token side by side
    qkv = _bf16(rng.standard_normal((b, n, h + 2 * hk, d))).cuda().transpose(1, 2)
    q, k, v = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
    pos = rng.integers(0, 1 << 20, (b, n)) if given else None
    if given:
        pos[0, 0] = (1 << 31) - 1
        pos[-1, -1] = -3
    freq = [10000.0 ** (-2.0 * i / rotary) for i in range(rotary // 2)]
    rope = wise.rope_frequencies(rotary, inv_freq=freq, pairs=pairs) if rotary else None
    got = wise.cache_append(cache, k, v, q=q if h else None, new_len=_i32(news), positions=_i32(pos), rope=rope)
    wise.check_device()
    kp, vp = C.append(_np(k0), _np(v0), table, lengths, _np(k), _np(v), news, pos, freq, pairs)
    assert np.array_equal(_np(cache.v_pages), vp)
    same = np.array_equal

    def near(x, want, size):
        return np.all(np.abs(x - want) <= BF16 * np.abs(want) + 2.0 ** -20 * size)
    big = np.abs(_np(k)).max() * 2
    written = kp != _np(k0)
    assert near(_np(cache.k_pages), kp, big)
    assert same(_np(cache.k_pages)[~written], _np(k0)[~written])
    if rotary < d:  # what is not rotated is copied
        assert same(_np(cache.k_pages)[..., rotary:], kp[..., rotary:])
    assert cache.lengths.tolist() == list(lengths)
    if not h:
        assert got is None
        return
    want = np.array(_np(q))
    for s in range(b):
        for i in range(n):
            for x in range(h):
                want[s, x, i] = C.rotate(want[s, x, i], lengths[s] + i if pos is None else pos[s, i], freq, pairs)
    assert got.shape == q.shape and got.is_contiguous()
    assert near(_np(got), want, np.abs(_np(q)).max() * 2)
    assert same(_np(got)[..., rotary:], want[..., rotary:])


def test_append_at_far_positions_is_exact():
    """The angle of a position near 2^31 is as exact as that of a near one."""
    d = 64
    pos = np.array([[0, 1, 10 ** 6 + 1, 2 ** 31 - 1, 2 ** 30 + 12345]])
    freq = [10000.0 ** (-2.0 * i / d) for i in range(d // 2)]
    x = np.zeros((1, 1, 5, d), np.float32)
    x[..., :d // 2] = 1.0  # keys (1, 0): rotated to (cos, sin)
    pool = torch.zeros((1, 1, 16, d), dtype=torch.bfloat16)
    cache = _cache(pool, pool, [[0]], [0])
    k = _bf16(x).cuda()
    wise.cache_append(cache, k, k, positions=_i32(pos), rope=wise.rope_frequencies(d, inv_freq=freq))
    wise.check_device()
    got = _np(cache.k_pages)[0, 0, :5]
    # frequencies are held to 2^-53 of a radian or better: at 2^31 that is 2^-22
    for i, p in enumerate(pos[0]):
        turns = [(int(p) * (int(round(f / (2 * np.pi) * 2.0 ** 64)) % (1 << 64))) % (1 << 64) / 2.0 ** 64 for f in freq]
        want = np.concatenate([np.cos(2 * np.pi * np.array(turns)), np.sin(2 * np.pi * np.array(turns))])
        assert np.all(np.abs(got[i] - want) <= BF16 * np.abs(want) + 2.0 ** -20)


# ------------------------------------------------------------------- accept

@pytest.mark.parametrize("case", [
    ([5], [3], [[0, 2, 5]], 1, 64, 16),
    ([0, 16, 31], [4, 1, 0], [[0, 1, 2, 3], [6, -1, -1, -1], [9, 9, 9, 9]], 2, 96, 16),
    ([100, 3], [20, 17], None, 3, 128, 32),       # long paths that overlap what they overwrite
    ([40, 7], [2, 5], "keep", 2, 128, 64),
], ids=["one", "ragged", "long", "no_path"])
def test_accept(case):
    lengths, kept, path, hk, d, page = case
    rng = np.random.default_rng(d)
    n = 40
    table, n_pages = _table(rng, [x + n for x in lengths], page)
    k, v = _bf16(rng.standard_normal((n_pages, hk, page, d))), _bf16(rng.standard_normal((n_pages, hk, page, d)))
    cache = _cache(k, v, table, lengths)
    if path is None:
        path = [sorted(rng.choice(n, 20, replace=False).tolist()) for _ in lengths]
    path = None if path == "keep" else path
    new = wise.cache_accept(cache, _i32(kept), _i32(path))
    wise.check_device()
    kp, vp, want = C.accept(_np(k), _np(v), table, lengths, kept, path)
    assert np.array_equal(_np(cache.k_pages), kp) and np.array_equal(_np(cache.v_pages), vp)
    assert new.tolist() == want.tolist() and cache.lengths.tolist() == list(lengths)


# ------------------------------------------------------- together, and graphs

def _speculate(cache, x, rope, steps):
    """Steps of drafting: append a tree, attend, keep a path."""
    outs = []
    for s in range(steps):
        k, v, q, pos_off, mask, kept, path, new_lengths = x[s]
        pos = cache.lengths[:, None] + pos_off
        q = wise.cache_append(cache, k, v, q=q, positions=pos, rope=rope)
        outs.append(wise.tree_attention(q, cache, tree_mask=mask))
        wise.cache_accept(cache, kept, path, new_lengths=new_lengths)
        cache.lengths.copy_(new_lengths)
    return outs


def _speculation(seed, b=2, h=4, hk=2, d=64, page=16, n=7, steps=3, prompt=40):
    rng = np.random.default_rng(seed)
    table, n_pages = _table(rng, [prompt + steps * n] * b, page)
    pool = torch.full((n_pages, hk, page, d), float("nan"), dtype=torch.bfloat16)
    cache = _cache(pool, pool, table, [0] * b)
    rope = wise.rope_frequencies(d)
    kv = _bf16(rng.standard_normal((2, b, hk, prompt, d))).cuda()
    x = []
    for _ in range(steps):
        sees = _tree(rng, b, n, "tree")
        path = np.full((b, n), -1)
        kept = []
        for s in range(b):
            leaf = int(rng.integers(0, n))
            line = np.nonzero(sees[s, leaf])[0]
            path[s, :len(line)] = line
            kept.append(len(line))
        k, v, q = (_bf16(rng.standard_normal((b, y, n, d))).cuda() for y in (hk, hk, h))
        x.append((k, v, q, _i32(sees.sum(2) - 1), wise.pack_tree_mask(torch.from_numpy(sees).cuda()), _i32(kept),
                  _i32(path), torch.zeros(b, dtype=torch.int32, device="cuda")))
    return cache, rope, kv, x, table


def test_drafting_loop_equals_a_plain_sequence():
    """Append, attention and acceptance together: the kept tokens of every
    step, as one plain sequence, give what each step's rows gave."""
    cache, rope, kv, x, table = _speculation(23)
    b, hk, prompt, d = kv.shape[1:]
    wise.cache_append(cache, kv[0], kv[1], rope=rope)
    cache.lengths = wise.cache_accept(cache, _i32([prompt] * b))
    seq = [[(_np(kv[0])[s, :, t], _np(kv[1])[s, :, t]) for t in range(prompt)] for s in range(b)]
    freq = [10000.0 ** (-2.0 * i / d) for i in range(d // 2)]
    outs = _speculate(cache, x, rope, len(x))
    wise.check_device()
    assert cache.lengths.tolist() == [prompt + sum(int(y[5][s]) for y in x) for s in range(b)]
    for (k, v, q, _, _, kept, path, _), (o, _) in zip(x, outs):
        for s in range(b):
            line = path[s, :int(kept[s])].tolist()
            for i in line:
                seq[s].append((_np(k)[s, :, i], _np(v)[s, :, i]))
                pos = len(seq[s]) - 1
                for y in range(q.shape[1]):
                    hh = y // (q.shape[1] // hk)
                    kk = np.array([C.rotate(z[0][hh], t, freq, False) for t, z in enumerate(seq[s])])
                    vv = np.array([z[1][hh] for z in seq[s]])
                    qq = C.rotate(_np(q)[s, y, i], pos, freq, False)
                    sc = kk @ qq / np.sqrt(d)
                    p = np.exp(sc - sc.max())
                    p /= p.sum()
                    want = p @ vv
                    # keys and queries were rounded to bf16 after their rotation: each
                    # score moves by at most 2 * 2^-8 of sum |q k|, and so do the weights
                    move = 2 * BF16 * (np.abs(kk) @ np.abs(qq)).max() / np.sqrt(d)
                    tol = (2 * BF16 + 2 * np.expm1(move)) * (p @ np.abs(vv)) + BF16 * np.abs(want) + 2.0 ** -16
                    assert np.all(np.abs(_np(o)[s, y, i] - want) <= tol)


def test_drafting_loop_replayed_from_a_graph():
    """The loop captured once and replayed gives the eager bits, and so does a
    second graph that is replayed between."""
    results = []
    for mode in ("eager", "graph"):
        cache, rope, kv, x, _ = _speculation(29)
        b, prompt = kv.shape[1], kv.shape[3]
        wise.cache_append(cache, kv[0], kv[1], rope=rope)
        cache.lengths = wise.cache_accept(cache, _i32([prompt] * b))
        start = [t.clone() for t in (cache.k_pages, cache.v_pages, cache.lengths)]
        if mode == "eager":
            outs = _speculate(cache, x, rope, len(x))
        else:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                _speculate(cache, x, rope, len(x))
            torch.cuda.current_stream().wait_stream(side)

            def back():
                for t, s in zip((cache.k_pages, cache.v_pages, cache.lengths), start):
                    t.copy_(s)
            graphs, kept = [], []
            for _ in range(2):
                back()
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    kept.append(_speculate(cache, x, rope, len(x)))
                graphs.append(g)
            for g in (graphs[0], graphs[1], graphs[0]):
                back()
                g.replay()
            outs = kept[0]
        torch.cuda.synchronize()
        wise.check_device()
        results.append((outs, cache.k_pages.clone(), cache.v_pages.clone(), cache.lengths.clone()))
    (eager, *a), (replayed, *r) = results
    for (o, lse), (o2, lse2) in zip(eager, replayed):
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert torch.equal(a[0].view(torch.int16), r[0].view(torch.int16)) and torch.equal(a[2], r[2])


FIRST_CALLS = """
import torch
import block_sparse_attention_causal_gb300 as wise
heads, n, d = %d, 3, 128
pool = torch.randn((8, 2, 16, d), device="cuda").bfloat16()
cache = wise.PagedCache(pool, pool.clone(), torch.arange(8, dtype=torch.int32, device="cuda").reshape(1, 8),
                        torch.tensor([40], dtype=torch.int32, device="cuda"))
q = torch.randn((1, heads, n, d), device="cuda").bfloat16()
k = torch.randn((1, 2, n, d), device="cuda").bfloat16()
kept, rope = torch.tensor([2], dtype=torch.int32, device="cuda"), wise.rope_frequencies(d)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    rotated = wise.cache_append(cache, k, k, q=q, rope=rope)
    o, lse = wise.tree_attention(rotated, cache)
    lengths = wise.cache_accept(cache, kept)
graph.replay()
torch.cuda.synchronize()
want = wise.tree_attention(rotated, cache)
assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and lengths.tolist() == [42]
wise.check_device()
"""


@pytest.mark.parametrize("heads", [8, 100])
def test_a_process_s_first_calls_are_captured(heads):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", FIRST_CALLS % heads], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr


def test_lengths_handed_from_call_to_call():
    """Each acceptance's lengths are the next call's, with no other kernel
    between them, and share their lines with the lengths that were read before."""
    rng = np.random.default_rng(53)
    b, h, hk, d, page, steps = 5, 8, 2, 64, 16, 24
    table, n_pages = _table(rng, [3 * steps] * b, page)
    kept = _i32(rng.integers(0, 4, (steps, b)))
    path = _i32([[0, 1, 2]] * b)
    x = [[_bf16(rng.standard_normal((b, y, 3, d))).cuda() for y in (h, hk, hk)] for _ in range(steps)]
    zero = torch.zeros((n_pages, hk, page, d), dtype=torch.bfloat16)
    rope = wise.rope_frequencies(d)
    results = []
    for wait in (True, False):
        lengths = _i32([[0] * b] + [[-1] * b] * steps)
        cache = _cache(zero, zero, table, [0] * b)
        outs = []
        torch.cuda.synchronize()
        for i, (q, k, v) in enumerate(x):
            cache.lengths = lengths[i]
            qr = wise.cache_append(cache, k, v, q=q, rope=rope)
            outs.append(wise.tree_attention(qr, cache, new_len=kept[i]))
            wise.cache_accept(cache, kept[i], path, new_lengths=lengths[i + 1])
            if wait:
                torch.cuda.synchronize()
        wise.check_device()
        assert torch.equal(lengths[1:], torch.cumsum(kept, 0).to(torch.int32))
        results.append((outs, cache.k_pages, cache.v_pages))
    for (o, lse), (o2, lse2) in zip(results[0][0], results[1][0]):
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert torch.equal(results[0][1], results[1][1]) and torch.equal(results[0][2], results[1][2])


def test_two_streams_at_once():
    rng = np.random.default_rng(31)
    want, got, made = [], [], []
    for i in range(2):
        lengths, page, d = [1500 + i, 40], 64, 128
        table, n_pages = _table(rng, [x + 1 for x in lengths], page)
        k, v = _pools(rng, 2, d, page, table, n_pages, [x + 1 for x in lengths])
        made.append((_cache(k, v, table, lengths), _bf16(rng.standard_normal((2, 8, 1, d))).cuda()))
        want.append(wise.tree_attention(made[i][1], made[i][0]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for s, (cache, q) in zip(streams, made):
            got.append(wise.tree_attention(q, cache, stream=s))
    torch.cuda.synchronize()
    wise.check_device()
    for j, (o, lse) in enumerate(got):
        assert torch.equal(o, want[j % 2][0]) and torch.equal(lse, want[j % 2][1])


def test_calls_on_given_streams_and_captured_forks():
    """Every call on a stream of its own, in order by events, and the same
    recorded into one graph whose branches run side by side."""
    rng = np.random.default_rng(47)
    lengths, page, d, h, hk, n = [200, 33], 32, 128, 8, 2, 5
    totals = [x + n for x in lengths]
    table, n_pages = _table(rng, totals, page)
    k, v = _pools(rng, hk, d, page, table, n_pages, totals, fill=0.0)
    x = [_bf16(rng.standard_normal((2, y, n, d))).cuda() for y in (hk, hk, h)]
    other = _cache(k, v, table, lengths)
    oq = _bf16(rng.standard_normal((2, h, 1, d))).cuda()
    rope = wise.rope_frequencies(d)
    kept, path = _i32([2, 3]), _i32([[0, 3, 0], [1, 2, 4]])

    def work(cache, a, b):
        """Append on one stream, attend on another (beside attention over
        another cache on the first), accept on the first again."""
        q = wise.cache_append(cache, x[0], x[1], q=x[2], rope=rope, stream=a)
        b.wait_stream(a)
        o, lse = wise.tree_attention(q, cache, stream=b)
        o2, lse2 = wise.tree_attention(oq, other, stream=a)
        a.wait_stream(b)
        return [q, o, lse, o2, lse2, wise.cache_accept(cache, kept, path, stream=a)]

    main = torch.cuda.current_stream()
    cache = _cache(k, v, table, lengths)
    want = work(cache, main, main)
    want += [cache.k_pages, cache.v_pages]
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    eager = _cache(k, v, table, lengths)
    a.wait_stream(main)
    got = work(eager, a, b)
    torch.cuda.synchronize()
    for u, w in zip(got + [eager.k_pages, eager.v_pages], want):
        assert torch.equal(u, w)
    again = _cache(k, v, table, lengths)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=a):
        got = work(again, a, b)
    for _ in range(3):
        again.k_pages.copy_(k)
        again.v_pages.copy_(v)
        for u in got:
            u.zero_()
        graph.replay()
        # eager calls on another stream meanwhile
        side, side_lse = wise.tree_attention(oq, other, stream=b)
        torch.cuda.synchronize()
        for u, w in zip(got + [again.k_pages, again.v_pages, side, side_lse], want + [want[3], want[4]]):
            assert torch.equal(u, w)
    wise.check_device()


# -------------------------------------------------------- entries that are bad

def test_bad_entries_are_flagged_and_skipped():
    rng = np.random.default_rng(37)
    lengths, page, d, n = [40, 20], 16, 64, 3
    table, n_pages = _table(rng, [43, 23], page, spare_cols=0)
    k, v = _pools(rng, 1, d, page, table, n_pages, [43, 23])
    q = _bf16(rng.standard_normal((2, 1, n, d))).cuda()
    sees = _tree(rng, 2, n, "run")

    def status():
        return wise.device_status()
    # a page outside the pool: its tokens are not seen, the rest is
    for bad in (-1, n_pages, 2 ** 30):
        t = table.copy()
        t[0, 1] = bad
        o, lse = wise.tree_attention(q, _cache(k, v, t, lengths), out_dtype=torch.float32)
        assert status() == _lib.WISE_ERR_BAD_CACHE and status() == _lib.WISE_OK
        # the same tokens from a cache that never held that page
        at = [x for x in range(43) if not 16 <= x < 32]
        dense_k, dense_v = (np.array([_np(p)[table[0][x // page], :, x % page] for x in at]) for p in (k, v))
        pool = np.zeros((2, 2, 1, page, d), np.float32)
        for x in range(len(at)):
            pool[0, x // page, :, x % page], pool[1, x // page, :, x % page] = dense_k[x], dense_v[x]
        want = wise.tree_attention(q[:1], _cache(_bf16(pool[0]), _bf16(pool[1]), [[0, 1]], [24]), out_dtype=torch.float32)
        assert status() == _lib.WISE_OK
        assert np.allclose(_np(o[:1]), _np(want[0]), atol=8 * BF16) and np.allclose(_np(lse[:1]), _np(want[1]), atol=1e-5)
    # counts outside their range
    good = _cache(k, v, table, lengths)
    for lens, news in (([-1, 20], [3, 3]), ([40, 20], [-1, 3]), ([40, 20], [4, 3]), ([48, 20], [3, 3]),
                       ([2 ** 31 - 1, 20], [3, 3])):
        c = wise.PagedCache(good.k_pages, good.v_pages, good.page_table, _i32(lens))
        o, lse = wise.tree_attention(q, c, new_len=_i32(news), out_dtype=torch.float32)
        assert status() == _lib.WISE_ERR_BAD_CACHE
        want, want_lse = wise.tree_attention(q, good, out_dtype=torch.float32)
        assert status() == _lib.WISE_OK
        assert torch.allclose(o[1], want[1], atol=8 * BF16) and torch.allclose(lse[1], want_lse[1], atol=1e-5)
        if news[0] == -1:
            assert torch.all(o[0] == 0) and torch.all(torch.isneginf(lse[0]))


def test_bad_entries_of_append_and_accept():
    rng = np.random.default_rng(41)
    page, d = 16, 64
    table = np.array([[0, 5], [1, 2]], np.int32)
    pool = _bf16(rng.standard_normal((3, 1, page, d)))
    x = _bf16(rng.standard_normal((2, 1, 20, d))).cuda()

    def run(lengths, news=None):
        c = _cache(pool, pool, table, lengths)
        wise.cache_append(c, x, x, new_len=_i32(news))
        return c
    c = run([0, 3])  # sequence 0's second page is not in the pool: 4 tokens skipped
    assert wise.device_status() == _lib.WISE_ERR_BAD_CACHE
    assert torch.equal(c.v_pages[0, 0], x[0, 0, :16]) and torch.equal(c.v_pages[1, 0, 3:], x[1, 0, :13])
    assert torch.equal(c.v_pages[2, 0, :7], x[1, 0, 13:]) and torch.equal(c.v_pages[2, 0, 7:].cpu(), pool[2, 0, 7:])
    for lengths, news in (([0, 13], [16, 20]), ([-1, 3], [1, 20]), ([0, 3], [16, 21]), ([0, 3], [-1, 20]),
                          ([0, 2 ** 31 - 1], [16, 20])):
        c = run(lengths, news)
        assert wise.device_status() == _lib.WISE_ERR_BAD_CACHE, (lengths, news)
        if lengths[0] == -1 or news[0] == -1:
            assert torch.equal(c.v_pages[0].cpu(), pool[0])
    # accepted paths: not ascending, past the table, a page outside the pool
    cache = _cache(pool, pool, table, [0, 3])
    for kept, path in (([2, 1], [[3, 3], [0, 0]]), ([1, 1], [[-2, 0], [0, 0]]), ([1, 2], [[0, 0], [0, 40]]),
                       ([1, 1], [[20, 0], [0, 0]]), ([3, 1], [[0, 1], [0, 0]]), ([-1, 1], [[0, 1], [0, 0]])):
        c = _cache(pool, pool, table, [0, 3])
        new = wise.cache_accept(c, _i32(kept), _i32(path))
        assert wise.device_status() == _lib.WISE_ERR_BAD_CACHE, (kept, path)
        assert new.tolist() == [max(0, min(kept[0], 2)), 3 + kept[1]]
        assert torch.equal(c.v_pages[1:].cpu(), pool[1:])
    new = wise.cache_accept(cache, _i32([0, 30]))  # only 29 slots are left
    assert wise.device_status() == _lib.WISE_ERR_BAD_CACHE and new.tolist() == [0, 32]


def test_calls_refuse_what_does_not_fit():
    rng = np.random.default_rng(43)
    pool = _bf16(rng.standard_normal((3, 2, 16, 64)))
    c = _cache(pool, pool, [[0, 1]], [4])
    x = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    for call in (
        lambda: wise.cache_append(c, x[:, :1], x),
        lambda: wise.cache_append(c, x, x[:, :, :2]),
        lambda: wise.cache_append(c, x.float(), x),
        lambda: wise.cache_append(c, x.transpose(2, 3), x),
        lambda: wise.cache_append(c, x, x, q=x[:, :, :2]),
        lambda: wise.cache_append(c, x, x, q_out=x),
        lambda: wise.cache_append(c, x, x, q=x, q_out=torch.empty((1, 2, 4, 64), dtype=torch.bfloat16, device="cuda")),
        lambda: wise.cache_append(c, x, x, new_len=torch.zeros(2, **i32)),
        lambda: wise.cache_append(c, x, x, new_len=torch.zeros(1, dtype=torch.int64, device="cuda")),
        lambda: wise.cache_append(c, x, x, positions=torch.zeros((1, 2), **i32)),
        lambda: wise.cache_append(c, x.cpu(), x),
        lambda: wise.tree_attention(x[:, :1], c),
        lambda: wise.tree_attention(x[..., :32], c),
        lambda: wise.tree_attention(x, c, tree_mask=torch.zeros((1, 3, 2), **i32)),
        lambda: wise.tree_attention(x, c, out_dtype=torch.float16),
        lambda: wise.tree_attention(x, c, out=torch.empty((1, 2, 3, 64), dtype=torch.float32, device="cuda")),
        lambda: wise.tree_attention(x, c, lse=torch.empty((1, 2, 2), dtype=torch.float32, device="cuda")),
        lambda: wise.tree_attention(x, c, workspace=torch.empty(8, dtype=torch.uint8, device="cuda")),
        lambda: wise.tree_attention(x, wise.PagedCache(c.k_pages, c.v_pages[:2], c.page_table, c.lengths)),
        lambda: wise.tree_attention(x, wise.PagedCache(c.k_pages, c.v_pages, c.page_table, c.lengths.long())),
        lambda: wise.tree_attention(x, wise.PagedCache(c.k_pages, c.v_pages, c.page_table.cpu(), c.lengths)),
        lambda: wise.tree_attention(x, wise.PagedCache(c.k_pages.transpose(0, 1), c.v_pages, c.page_table, c.lengths)),
        lambda: wise.cache_accept(c, torch.zeros(2, **i32)),
        lambda: wise.cache_accept(c, torch.zeros(1, **i32), torch.zeros((2, 3), **i32)),
        lambda: wise.cache_accept(c, torch.zeros(1, **i32), torch.zeros(3, **i32)),
    ):
        with pytest.raises(ValueError):
            call()
    for call in (
        lambda: wise.cache_append(c, x, x, rope=wise.rope_frequencies(128)),
        lambda: wise.cache_append(c, torch.zeros((1, 2, 3, 68), dtype=torch.bfloat16, device="cuda")[..., :64], x),
        lambda: wise.cache_append(c, torch.zeros(400, dtype=torch.bfloat16, device="cuda")[1:385].view(1, 2, 3, 64), x),
        lambda: wise.tree_attention(torch.zeros((1, 2, 129, 64), dtype=torch.bfloat16, device="cuda"), c),
        lambda: wise.tree_attention(x, c, scale=-1.0),
        lambda: wise.cache_accept(c, torch.zeros(1, **i32), new_lengths=c.lengths),
    ):
        with pytest.raises(wise.WiseError):
            call()
    wise.check_device()
