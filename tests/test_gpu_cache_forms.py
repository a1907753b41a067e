"""The paged-cache operators on the GPU in the forms that differ in code:
rotations at every size of angle, every instance of the attention kernels, pages
outside the pool under each of them, long prompts and long accepted paths.

Tolerances. A rounding to bf16 is off by at most 2^-8 of the value, one in fp32
by 2^-24.
 * rotation: the sine and cosine are good to 2^-22 of their value; the two
   products and their sum add 2^-24 each, so a result is off by less than 2^-21
   of |x cos a| + |y sin a| before its one rounding to bf16 (times 1 + 2^-21).
 * attention: a score is a sum of exact products in fp32, off by at most
   e_s = (d + 8) 2^-24 * scale * sum |q k|, the scale's own rounding among them;
   its exponential adds 2^-22. A weight is rounded to bf16 (2^-8) in the numerator
   only; the sum that divides it is of the fp32 values. Sums in fp32: of the
   numerator, at most 16 steps a tile of 128 tokens and one addition for each
   of at most 152 parts, 2^-23 each (a tensor core may cut off); of the
   divisor, at most 40 additions, one a tile and one a part. So O is off by at
   most (2^-8 + 2 e_s + 2^-20 + 2^-23 (17 tiles + 400)) * sum a |v|, 1 % more
   for products of these terms, plus 2^-8 of it where O is rounded to bf16.
 * LSE: e_s, 2^-20 for the exponential and the logarithm, 2^-24 for each of the
   divisor's additions, and 2^-22 of its value.
"""
import math

import numpy as np
import pytest
import torch

import block_sparse_attention_causal_gb300 as wise
from block_sparse_attention_causal_gb300 import _lib
from oracle import cache_oracle as C

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


def test_one_pool_for_keys_and_values_is_read_but_not_written():
    g = torch.Generator(device="cuda").manual_seed(6)
    pool = torch.randn((4, 2, 16, 64), generator=g, device="cuda").bfloat16()
    tied = wise.PagedCache(pool, pool, _i32([[2, 0], [1, 3]]), _i32([20, 5]))
    apart = wise.PagedCache(pool, pool.clone(), tied.page_table, tied.lengths)
    before = pool.clone()
    q = torch.randn((2, 4, 2, 64), generator=g, device="cuda").bfloat16()
    for got, want in zip(wise.tree_attention(q, tied), wise.tree_attention(q, apart)):
        assert torch.equal(got, want)
    assert wise.cache_accept(tied, _i32([2, 0])).tolist() == [22, 5]  # moves nothing
    with pytest.raises(wise.WiseError):
        wise.cache_accept(tied, _i32([2, 0]), _i32([[0, 1], [0, 0]]))
    with pytest.raises(wise.WiseError):
        wise.cache_append(tied, q[:, :2], q[:, 2:])
    wise.check_device()
    assert torch.equal(pool, before)


# ---------------------------------------------------------------- attention

def _paged(g, totals, hk, d, page, spare_cols=1, spare_pages=2):
    """Random keys and values in every token's row, NaN in all others; pages
    handed out in random order, entries past a sequence's last token -1."""
    used = [max(1, (t + page - 1) // page) for t in totals]
    n_pages = sum(used) + spare_pages
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(totals), max(used) + spare_cols), -1, dtype=torch.int32, device="cuda")
    k, v = (torch.randn((n_pages, hk, page, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    spare = torch.ones(n_pages, dtype=torch.bool, device="cuda")
    at = 0
    for b, (u, t) in enumerate(zip(used, totals)):
        table[b, :u] = order[at:at + u]
        at += u
        spare[table[b, :u].long()] = False
        last = int(table[b, u - 1])
        k[last, :, t - (u - 1) * page:] = float("nan")
        v[last, :, t - (u - 1) * page:] = float("nan")
    k[spare], v[spare] = float("nan"), float("nan")
    return k, v, table


def _sees(g, b, n, kind):
    if kind == "run":
        return torch.ones((n, n), dtype=torch.bool, device="cuda").tril().expand(b, n, n)
    m = torch.rand((b, n, n), generator=g, device="cuda") < 0.4
    m[:, n // 2] = False  # a token that sees nothing new
    return m


def _check_attention(q, cache, sees, lengths, news, dtype=torch.float32, mask=None, missing=(), status=_lib.WISE_OK):
    """tree_attention against the formula in 64 bits. missing: (sequence, column
    of the page table) whose tokens nobody sees."""
    b, h, n, d = q.shape
    hk, page = cache.k_pages.shape[1], cache.k_pages.shape[2]
    o, lse = wise.tree_attention(q, cache, new_len=None if news is None else _i32(news), tree_mask=mask, out_dtype=dtype)
    assert wise.device_status() == status
    again = wise.tree_attention(q, cache, new_len=None if news is None else _i32(news), tree_mask=mask, out_dtype=dtype)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])  # joined in a fixed order
    assert wise.device_status() == status
    for s in range(b):
        m = n if news is None else news[s]
        total = lengths[s] + m
        assert torch.all(o[s, :, m:] == 0) and torch.all(torch.isneginf(lse[s, :, m:]))
        if m == 0:
            continue
        gone = torch.zeros(max(total, 1), dtype=torch.bool, device="cuda")[:total]
        cols = cache.page_table[s, :(total + page - 1) // page].long().clone()
        for x, col in missing:
            if x == s:
                gone[col * page:(col + 1) * page] = True
                cols[col] = 0
        kk, vv = (p[cols].transpose(0, 1).reshape(hk, -1, d)[:, :total].double() for p in (cache.k_pages, cache.v_pages))
        kk, vv = kk.masked_fill(gone[None, :, None], 0.0), vv.masked_fill(gone[None, :, None], 0.0)
        seen = torch.cat([torch.ones((m, lengths[s]), dtype=torch.bool, device="cuda"), sees[s][:m, :m]], 1) & ~gone
        qq = q[s, :, :m].double().reshape(hk, h // hk * m, d)
        sc = (qq @ kk.transpose(1, 2) / math.sqrt(d)).reshape(h, m, total).masked_fill(~seen, -math.inf)
        size = (qq.abs() @ kk.abs().transpose(1, 2) / math.sqrt(d)).reshape(h, m, total).masked_fill(~seen, 0.0).amax(-1)
        want_lse = torch.logsumexp(sc, -1)
        some = seen.any(-1)
        a = torch.exp(sc - torch.where(some, want_lse, 0.0)[..., None])
        a = a.reshape(hk, -1, total)
        want, weight = (a @ vv).reshape(h, m, d), (a @ vv.abs()).reshape(h, m, d)
        tiles = (total + 127) // 128
        e_s = ((d + 8) * F32 * size)[..., None]
        tol = 1.01 * (BF16 + 2 * e_s + 2.0 ** -20 + 2.0 ** -23 * (17 * tiles + 400)) * weight
        if dtype == torch.bfloat16:
            tol = tol + BF16 * (want.abs() + tol)
        got = o[s, :, :m].double()
        assert torch.isfinite(got).all()
        assert torch.all((got - want).abs() <= tol), float(((got - want).abs() / tol.clamp(min=1e-30)).max())
        off = (lse[s, :, :m].double() - want_lse).abs()
        tol = e_s[..., 0] + 2.0 ** -20 + F32 * (192 + tiles) + 2.0 ** -22 * want_lse.abs()
        assert torch.all(off[:, some] <= tol[:, some])
        assert torch.all(got[:, ~some] == 0) and torch.all(torch.isneginf(lse[s, :, :m][:, ~some]))
    return o, lse


# heads, key heads, new tokens: up to 16, 32, 64, 128 and 256 rows of a key head, and more
ROWS = {"16": (8, 2, 3), "32": (8, 2, 7), "64": (6, 2, 19), "128": (10, 2, 20), "256": (8, 2, 61), "more": (6, 2, 101)}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("d", [64, 96, 128])
def test_every_kernel_over_ragged_sequences(d, rows, dtype):
    """Empty and one-token caches, both sides of a tile's end, sequences without
    new tokens, masks that leave a row nothing."""
    h, hk, n = ROWS[rows]
    g = torch.Generator(device="cuda").manual_seed(1000 * d + n)
    lengths = [0, 1, 127, 128, 129, 300, 64, 0]
    news = [n, 1, n, 0, (n + 1) // 2, n, max(1, n - 1), 0]
    for kind, page in (("run", 32), ("random", 64)):
        k, v, table = _paged(g, [x + y for x, y in zip(lengths, news)], hk, d, page)
        cache = wise.PagedCache(k, v, table, _i32(lengths))
        q = (torch.randn((len(lengths), h, n, d), generator=g, device="cuda") * 1.5).bfloat16()
        sees = _sees(g, len(lengths), n, kind)
        _check_attention(q, cache, sees, lengths, news, dtype, None if kind == "run" else wise.pack_tree_mask(sees))


@pytest.mark.parametrize("hk", [4, 1])
@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("d", [64, 96, 128])
def test_every_kernel_over_long_sequences(d, rows, hk):
    """Blocks that work through more key tiles than their rings hold: with 4 key
    heads, 160 units or more, whose partial results are found by block; with one,
    a few units, found by unit, in many parts each."""
    h, of, n = ROWS[rows]
    h = h // of * hk
    g = torch.Generator(device="cuda").manual_seed(d + n + hk)
    b = 40 if hk == 4 else 2
    lengths = torch.randint(1500, 2500, (b,), generator=g, device="cuda").tolist() if hk == 4 else [70000, 66001]
    news = [n - (i % 3) * (n // 3) for i in range(b)]
    k, v, table = _paged(g, [x + y for x, y in zip(lengths, news)], hk, d, 128 if d == 64 else 32)
    cache = wise.PagedCache(k, v, table, _i32(lengths))
    q = torch.randn((b, h, n, d), generator=g, device="cuda").bfloat16()
    sees = _sees(g, b, n, "random")
    _check_attention(q, cache, sees, lengths, news, mask=wise.pack_tree_mask(sees))


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("rows", list(ROWS))
@pytest.mark.parametrize("d", [64, 128])
def test_pages_outside_the_pool_are_not_seen(d, rows, page):
    """The first, a middle and the last page of a tile, the page of the drafted
    tokens and all of a sequence's pages, in pools whose other pages are NaN."""
    h, hk, n = ROWS[rows]
    g = torch.Generator(device="cuda").manual_seed(d + n + page)
    lengths = [700, 256, 1, 900]
    totals = [x + n for x in lengths]
    k, v, table = _paged(g, totals, hk, d, page)
    n_pages, per = k.shape[0], 128 // page
    missing = [(0, 0), (0, per + per // 2), (0, 3 * per - 1), (1, 256 // page), (2, 0)]
    missing += [(2, c) for c in range(1, (totals[2] + page - 1) // page)]
    for i, (s, col) in enumerate(missing):
        if int(table[s, col]) >= 0:  # what it held is spoilt, so that reading it would show
            k[int(table[s, col])], v[int(table[s, col])] = float("nan"), float("nan")
        table[s, col] = (-1, n_pages, 2 ** 31 - 1, -2 ** 31)[i % 4]
    cache = wise.PagedCache(k, v, table, _i32(lengths))
    q = torch.randn((4, h, n, d), generator=g, device="cuda").bfloat16()
    for kind in ("run", "random"):
        sees = _sees(g, 4, n, kind)
        _check_attention(q, cache, sees, lengths, None, mask=None if kind == "run" else wise.pack_tree_mask(sees),
                         missing=missing, status=_lib.WISE_ERR_BAD_CACHE)


# ------------------------------------------------------ long prompts and paths

def _rotated(x, pos, steps, pairs):
    """(x rotated, |x cos a| + |y sin a|) in 64 bits; x [b, heads, n, d], pos [b, n]."""
    half = len(steps)
    if half == 0:
        return x, torch.zeros_like(x)
    step = torch.tensor([t - (1 << 64) if t >> 63 else t for t in steps], dtype=torch.int64, device="cuda")
    at = pos.long()[..., None] * step + (1 << 61)  # modulo 2^64
    rest = ((at & ((1 << 62) - 1)) - (1 << 61)).double() * (math.pi * 2.0 ** -63)
    quarter = (at >> 62) & 3
    c0, s0 = torch.cos(rest), torch.sin(rest)
    c = torch.where(quarter == 0, c0, torch.where(quarter == 1, -s0, torch.where(quarter == 2, -c0, s0)))[:, None]
    s = torch.where(quarter == 0, s0, torch.where(quarter == 1, c0, torch.where(quarter == 2, -s0, -c0)))[:, None]
    i, j = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if pairs else (slice(0, half), slice(half, 2 * half))
    y, size = x.clone(), torch.zeros_like(x)
    y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., j] * c + x[..., i] * s
    size[..., i] = (x[..., i] * c).abs() + (x[..., j] * s).abs()
    size[..., j] = (x[..., j] * c).abs() + (x[..., i] * s).abs()
    return y, size


LONG = [  # sequences, tokens, heads (0: no q), key heads, d, page, rotary, neighbouring pairs
    (1, 4100, 32, 8, 128, 128, 128, False), (2, 13001, 5, 3, 64, 64, 64, True), (3, 6101, 5, 3, 96, 32, 48, False),
    (1, 17501, 5, 3, 96, 16, 96, True), (2, 6601, 5, 3, 128, 16, 96, False), (1, 9801, 0, 8, 128, 64, 128, True),
    (1, 26500, 7, 2, 64, 128, 32, False),
]


@pytest.mark.parametrize("case", LONG, ids=lambda c: "b%d_n%d_h%d_%d_d%d_p%d_r%d_%s" % (*c[:7], "pairs" if c[7] else "halves"))
def test_append_of_long_prompts(case):
    """Threads that keep four heads in flight: counts of heads that four does
    not divide, sequences that end early, a page outside the pool (its tokens
    are skipped, their queries rotated all the same), every other slot as it was."""
    b, n, h, hk, d, page, rotary, pairs = case
    g = torch.Generator(device="cuda").manual_seed(n)
    lengths = [(0, 37, 128)[i % 3] + 5 * i for i in range(b)]
    news = [n - i * (n // 5) - 1 for i in range(b)]
    k0, v0, table = _paged(g, [x + y for x, y in zip(lengths, news)], hk, d, page)
    k0, v0 = torch.nan_to_num(k0), torch.nan_to_num(v0)
    good = wise.PagedCache(k0.clone(), v0.clone(), table, _i32(lengths))
    qkv = torch.randn((b, n, h + 2 * hk, d), generator=g, device="cuda").bfloat16().transpose(1, 2)
    q, k, v = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
    freq = [500000.0 ** (-2.0 * i / max(rotary, 1)) for i in range(rotary // 2)]
    rope = wise.rope_frequencies(rotary, inv_freq=freq, pairs=pairs)
    pos = _i32(lengths)[:, None] + torch.arange(n, dtype=torch.int32, device="cuda")
    want, size = _rotated(qkv[:, :h + hk].double(), pos, _steps(freq), pairs)
    limit = BF16 * want.abs() + (1 + BF16) * 2.0 ** -21 * size
    limit[..., rotary:] = 0.0
    for bad_col in (None, (lengths[0] + news[0]) // page // 2):
        cache = wise.PagedCache(good.k_pages.clone(), good.v_pages.clone(), table.clone(), good.lengths)
        if bad_col is not None:
            cache.page_table[0, bad_col] = k0.shape[0]
        got = wise.cache_append(cache, k, v, q=q if h else None, new_len=_i32(news), rope=rope)
        assert wise.device_status() == (_lib.WISE_OK if bad_col is None else _lib.WISE_ERR_BAD_CACHE)
        if h:
            assert torch.all((got.double() - want[:, :h]).abs() <= limit[:, :h])
        else:
            assert got is None
        kp, vp, lim = k0.double(), v0.clone(), torch.zeros(k0.shape, dtype=torch.float64, device="cuda")
        for s in range(b):
            slot = lengths[s] + torch.arange(news[s], device="cuda")
            i = torch.arange(news[s], device="cuda")
            if s == 0 and bad_col is not None:
                keep = slot // page != bad_col
                slot, i = slot[keep], i[keep]
            pg, row = table[s].long()[slot // page], slot % page
            kp[pg, :, row] = want[s][h:][:, i].transpose(0, 1)
            lim[pg, :, row] = limit[s][h:][:, i].transpose(0, 1)
            vp[pg, :, row] = v[s][:, i].transpose(0, 1)
        assert torch.all((cache.k_pages.double() - kp).abs() <= lim)  # (0 where nothing is rotated or written)
        assert torch.equal(cache.v_pages, vp)


@pytest.mark.parametrize("kept", [129, 256, 300])
def test_accept_of_long_paths(kept):
    """More kept tokens than a block looks up at a time, each moved over slots
    that later ones are read from."""
    lengths, hk, d, page, n = [77, 0, 1000], 2, 96, 16, 512
    g = torch.Generator(device="cuda").manual_seed(kept)
    k, v, table = _paged(g, [x + n for x in lengths], hk, d, page)
    k, v = torch.nan_to_num(k), torch.nan_to_num(v)
    rng = np.random.default_rng(kept)
    counts = [kept, kept - 1, 128]
    path = np.full((3, kept), -1)
    for s, c in enumerate(counts):
        path[s, :c] = np.sort(rng.choice(n, c, replace=False)) if s != 1 else np.arange(1, c + 1)
    cache = wise.PagedCache(k.clone(), v.clone(), table, _i32(lengths))
    new = wise.cache_accept(cache, _i32(counts), _i32(path))
    wise.check_device()
    kp, vp, want = C.accept(k.float().cpu().numpy(), v.float().cpu().numpy(), table.cpu().numpy(), lengths, counts, path)
    assert np.array_equal(_np(cache.k_pages), kp) and np.array_equal(_np(cache.v_pages), vp)
    assert new.tolist() == want.tolist()


def test_moves_past_32_bits():
    """Keys and values that are kept in pages whose elements lie past 2^32."""
    page, d, hk = 128, 128, 2
    n_pages = (1 << 32) // (page * d * hk) + 8
    k, v = (torch.empty((n_pages, hk, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = np.array([[n_pages - 1, n_pages - 3], [n_pages - 5, n_pages - 2]])
    cache = wise.PagedCache(k, v, _i32(table), _i32([0, 0]))
    g = torch.Generator(device="cuda").manual_seed(9)
    x, y = (torch.randn((2, hk, 200, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    wise.cache_append(cache, x, y)
    cache.lengths = _i32([120, 130])
    new = wise.cache_accept(cache, _i32([4, 3]), _i32([[1, 4, 20, 60], [0, 2, 3, -1]]))
    wise.check_device()
    assert new.tolist() == [124, 133]
    keep = [list(range(120)) + [121, 124, 140, 180], list(range(130)) + [130, 132, 133]]
    for s in range(2):
        pages = torch.tensor(table[s], device="cuda")
        for pool, rows in ((k, x), (v, y)):
            got = pool[pages].transpose(0, 1).reshape(hk, -1, d)[:, :len(keep[s])]
            assert torch.equal(got, rows[s][:, keep[s]])


def test_two_graphs_of_the_loop_replayed_in_turn():
    """Append, attention and acceptance captured twice, replayed in turn and over
    again: each graph's own results are the eager ones, keys and values too."""
    b, h, hk, n, d, page = 2, 8, 2, 5, 64, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    lengths = [40, 300]
    k0, v0, table = _paged(g, [x + 2 * n for x in lengths], hk, d, page)
    k0, v0 = torch.nan_to_num(k0), torch.nan_to_num(v0)
    q, k, v = (torch.randn((b, x, n, d), generator=g, device="cuda").bfloat16() for x in (h, hk, hk))
    sees = _sees(g, b, n, "random")
    mask, rope = wise.pack_tree_mask(sees), wise.rope_frequencies(d)
    kept, path, start = _i32([3, 2]), _i32([[0, 2, 4], [1, 3, -1]]), _i32(lengths)
    cache = wise.PagedCache(k0.clone(), v0.clone(), table, start.clone())

    def back():
        cache.k_pages.copy_(k0)
        cache.v_pages.copy_(v0)
        cache.lengths.copy_(start)

    def loop():
        out = []
        for _ in range(2):
            r = wise.cache_append(cache, k, v, q=q, rope=rope)
            out += [r, *wise.tree_attention(r, cache, tree_mask=mask)]
            new = wise.cache_accept(cache, kept, path)
            cache.lengths.copy_(new)
            out.append(new)
        return out
    want = [x.clone() for x in loop() + [cache.k_pages, cache.v_pages]]
    graphs = []
    for _ in range(2):
        back()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = loop()
        graphs.append((graph, out))
    for i in (0, 1, 1, 0):
        back()
        for x in graphs[i][1]:
            x.zero_()
        graphs[i][0].replay()
        torch.cuda.synchronize()
        for x, y in zip(graphs[i][1] + [cache.k_pages, cache.v_pages], want):
            assert torch.equal(x, y)
    wise.check_device()
