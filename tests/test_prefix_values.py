"""Values of shared-prefix attention, element by element, where attention is sharp
enough that every tile of values shows: against the formula in 64 bits over the
whole length.

With keys of standard deviation 1 and queries of 3, scores have a deviation of
3: of 16K keys some 30 have a weight above 0.004 each, so each tile of 128
matters to some row. The bounds are those of the attention over a cache: a score
is off by e_s = (d + 8) 2^-24 scale sum |q k|; a weight is rounded to bf16, 2^-8,
in the numerator and in the sum alike; LSE by e_s, 2^-20, and 2^-24 for each
addition of the longest chain and of its value, which shifts a part's share of O
by as much, relative to it; the join's exponentials and logarithm 2^-20 more. O's
bound is that share of sum a |v| of its row and dimension. The CPU test plants
wrong tiles in the formula and shows that the bound finds each: they move O by
more than twice the bound, whatever the kernel's own error."""
import math

import numpy as np
import pytest
import torch

import block_sparse_attention_causal_gb300 as wise

gpu = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]
BF16, F32, TILE = 2.0 ** -8, 2.0 ** -24, 128


class Batch:
    """Groups of `members` sequences behind a shared prefix each, on the CPU: the
    tokens of the page in which the prefix ends stand in each sequence's own."""

    def __init__(self, seed, d, h, hk, n, groups, members, prefix, own, page, sharp=3.0):
        rng = np.random.default_rng(seed)
        b, whole, tail = groups * members, prefix // page, (own + page - 1) // page + 1
        self.page, self.prefix, self.groups, self.members = page, prefix, groups, members
        order = torch.from_numpy(rng.permutation(groups * whole + b * tail).astype(np.int32))
        shared = order[:groups * whole].reshape(groups, whole).repeat_interleave(members, 0)
        self.table = torch.cat([shared, order[groups * whole:].reshape(b, tail)], 1).contiguous()

        def draw(*shape, scale=1.0):
            return (torch.from_numpy(rng.standard_normal(shape, dtype=np.float32)) * scale).to(torch.bfloat16)
        self.k, self.v = (draw(order.numel(), hk, page, d) for _ in range(2))
        left = prefix % page
        for s in range(b):
            first = s // members * members
            if left and s != first:
                for p in (self.k, self.v):
                    p[int(self.table[s, whole]), :, :left] = p[int(self.table[first, whole]), :, :left]
        self.lengths = (prefix + torch.from_numpy(rng.integers(0, own - n, b))).to(torch.int32)
        self.q = draw(b, h, n, d, scale=sharp)

    def to(self, device):
        for name in ("table", "k", "v", "lengths", "q"):
            setattr(self, name, getattr(self, name).to(device))
        return self

    def cache(self):
        return wise.PagedCache(self.k, self.v, self.table, self.lengths)

    def groups_of(self):
        return (torch.full((self.groups,), self.prefix, dtype=torch.int32, device=self.q.device),
                (torch.arange(self.groups + 1, device=self.q.device) * self.members).to(torch.int32))

    def sequence(self, s):
        """Keys and values [kv_heads, tokens, d] of sequence s and who sees them
        [n, tokens], in 64 bits; tokens of pages outside the pool are not seen."""
        n, length = self.q.shape[2], int(self.lengths[s])
        t = torch.arange(length + n, device=self.q.device)
        pages = self.table[s].long()[t // self.page]
        there = (pages >= 0) & (pages < self.k.shape[0])
        pages = torch.where(there, pages, 0)
        k, v = (p[pages, :, t % self.page].double().transpose(0, 1) for p in (self.k, self.v))
        sees = there & (t <= length + torch.arange(n, device=t.device)[:, None])  # a run: tokens 0 .. i
        return k, v, sees

    def exact(self, s, heads=None):
        """(O, LSE, bound on O, bound on LSE, weights, values) of sequence s, rows
        [kv_heads, group, n]."""
        k, v, sees = self.sequence(s)
        if heads is not None:
            k, v = k[:heads], v[:heads]
        h, n, d = self.q.shape[1:]
        hk, group, scale = k.shape[0], h // self.k.shape[1], 1.0 / math.sqrt(d)
        q = self.q[s, :hk * group].double().reshape(hk, group, n, d)
        score = torch.einsum("xgnd,xtd->xgnt", q, k) * scale
        score = torch.where(sees, score, -math.inf)
        lse = torch.logsumexp(score, -1)
        p = torch.exp(score - lse[..., None])
        o, size_v = torch.einsum("xgnt,xtd->xgnd", p, v), torch.einsum("xgnt,xtd->xgnd", p, v.abs())
        size = torch.einsum("xgnd,xtd->xgnt", q.abs(), k.abs()).amax(-1) * scale
        e_s = (d + 8) * F32 * size
        part = e_s + 2.0 ** -20 + F32 * (64 + k.shape[1] / 8 + 2 * lse.abs())
        tol = (2 * BF16 + 2 * e_s + 2 * part + 2.0 ** -19)[..., None] * size_v
        return o, lse, tol, part + 2.0 ** -20 + F32 * 2 * lse.abs(), p, v


def _compare(batch, o, lse):
    b, h, n, d = batch.q.shape
    for s in range(b):
        want, want_lse, tol, lse_tol, _, _ = batch.exact(s)
        off = (o[s].double() - want.reshape(h, n, d)).abs() - tol.reshape(h, n, d)
        assert float(off.max()) <= 0.0, f"O of sequence {s}: {float(off.max()):.3e} past the bound"
        off = (lse[s].double() - want_lse.reshape(h, n)).abs() - lse_tol.reshape(h, n)
        assert float(off.max()) <= 0.0, f"LSE of sequence {s}: {float(off.max()):.3e} past the bound"


# d, heads, key heads, new tokens, members: 256, 64 and 600 rows of a group and key head
LONG = [(128, 32, 8, 1, 64), (64, 8, 2, 2, 8), (96, 40, 8, 5, 24)]


def _long(d, h, hk, n, members):
    return Batch(5, d, h, hk, n, 1, members, 16411, 5 * 64, 64)


@pytest.mark.parametrize("d,h,hk,n,members", LONG)
def test_the_bound_finds_every_wrong_tile(d, h, hk, n, members):
    """The formula with the values of one tile of the prefix taken from the tile
    behind it, or left out: for each tile some row's O is off by more than twice
    its bound."""
    batch = _long(d, h, hk, n, members)
    tiles = batch.prefix // TILE
    swapped, gone = torch.zeros(tiles, dtype=torch.float64), torch.zeros(tiles, dtype=torch.float64)
    for s in range(members):
        _, _, tol, _, p, v = batch.exact(s, heads=1)
        x = v[0, :tiles * TILE].reshape(tiles, TILE, d)
        w = p[0].reshape(-1, p.shape[-1])[:, :tiles * TILE].reshape(-1, tiles, TILE)
        tol = tol.reshape(-1, 1, d)
        here, behind = torch.einsum("rtk,tkd->rtd", w, x), torch.einsum("rtk,tkd->rtd", w, x.roll(-1, 0))
        swapped = torch.maximum(swapped, ((behind - here).abs() / tol).amax((0, 2)))
        gone = torch.maximum(gone, (here.abs() / tol).amax((0, 2)))
    assert float(swapped.min()) > 2.0 and float(gone.min()) > 2.0, (float(swapped.min()), float(gone.min()))


@pytest.mark.parametrize("d,h,hk,n,members", [pytest.param(*x, marks=gpu) for x in LONG])
def test_long_prefixes(d, h, hk, n, members):
    """Units cut over many blocks, rings gone round, in wide and narrow kernels."""
    batch = _long(d, h, hk, n, members).to("cuda")
    pre, _ = batch.groups_of()
    o, lse = wise.prefix_attention(batch.q, batch.cache(), pre, out_dtype=torch.float32)
    wise.check_device()
    _compare(batch, o, lse)


# 5 or 3 sequences a group: with its size said (narrow units, of rows that are no whole
# blocks) and not (wide ones), more groups than SMs and fewer
@pytest.mark.parametrize("d,h,hk,n,groups,members,prefix",
                         [pytest.param(*x, marks=gpu) for x in
                          [(64, 4, 1, 1, 260, 5, 256), (128, 8, 2, 3, 40, 3, 1300), (96, 12, 4, 7, 9, 5, 2050)]])
def test_many_groups(d, h, hk, n, groups, members, prefix):
    batch = Batch(6, d, h, hk, n, groups, members, prefix, 40, 16).to("cuda")
    pre, starts = batch.groups_of()
    for most in (0, members):
        o, lse = wise.prefix_attention(batch.q, batch.cache(), pre, group_starts=starts, max_members=most, out_dtype=torch.float32)
        wise.check_device()
        _compare(batch, o, lse)


@pytest.mark.parametrize("d,h,hk,n,members", [pytest.param(*x, marks=gpu) for x in [(64, 4, 2, 1, 6), (128, 16, 2, 4, 5), (96, 8, 1, 9, 4)]])
def test_shared_pages_outside_the_pool(d, h, hk, n, members):
    """Their tokens are seen by no row; the others' weights and values are what
    they are without them."""
    batch = Batch(7, d, h, hk, n, 1, members, 1030, 40, 32)
    batch.table[:, 3] = batch.k.shape[0]
    batch.table[:, 17:19] = -1
    batch.to("cuda")
    pre, _ = batch.groups_of()
    o, lse = wise.prefix_attention(batch.q, batch.cache(), pre, out_dtype=torch.float32)
    assert wise.device_status() == wise._lib.WISE_ERR_BAD_CACHE
    _compare(batch, o, lse)
