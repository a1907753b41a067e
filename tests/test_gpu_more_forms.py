"""Norms with rotation, shared prefixes, gathered weights and eviction on the GPU:
every kernel instance, graphs, streams, calls one after the other, far offsets.
Results are compared with the formulas in 64 bits within the bounds of the
operators' own tests, or bit for bit with another run of the same arithmetic."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import block_sparse_attention_causal_gb300 as wise
from tests.test_gpu_prefix import _bf16, _check, _i32, _mask, _shared_cache

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


def _randn(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


# sequences, new tokens and heads: 8, 28, 60, 120 and 300 rows of the group, the
# own parts in narrow and wide units
@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("b,n,h,hk", [(2, 1, 4, 1), (7, 1, 8, 2), (5, 6, 2, 1), (6, 20, 1, 1), (4, 25, 6, 2), (2, 70, 2, 2)])
def test_every_instance_of_the_shared_part(d, b, n, h, hk):
    rng = np.random.default_rng(b * 1000 + d)
    page = {64: 16, 96: 32, 128: 64}[d]
    prefix, lengths = 330, [330 + (37 * s) % 150 for s in range(b)]
    cache, table = _shared_cache(rng, [0, b], [prefix], lengths, [n] * b, hk, d, page)
    q = _bf16(rng.standard_normal((b, h, n, d)) * 1.5)
    sees, mask = _mask(rng, b, n, "random" if n > 2 else "run")
    got = wise.prefix_attention(q, cache, _i32([prefix]), tree_mask=mask, out_dtype=torch.float32)
    wise.check_device()
    _check(q, cache, table, sees, lengths, [n] * b, got, torch.float32)


def test_many_sequences_in_many_groups():
    """More groups than SMs, more sequences than a block's threads; against the
    attention without sharing."""
    g = torch.Generator(device="cuda").manual_seed(2)
    groups, members, hk, d, page, prefix = 260, 5, 1, 64, 16, 256
    b, whole = groups * members, prefix // page
    table = torch.full((b, whole + 2), -1, dtype=torch.int32, device="cuda")
    table[:, :whole] = torch.arange(groups * whole, device="cuda", dtype=torch.int32).reshape(groups, whole).repeat_interleave(members, 0)
    table[:, whole] = groups * whole + torch.arange(b, device="cuda", dtype=torch.int32)
    k, v = (_randn(g, groups * whole + b, hk, page, d) for _ in range(2))
    lengths = prefix + torch.randint(0, page - 2, (b,), generator=g, device="cuda").to(torch.int32)
    cache = wise.PagedCache(k, v, table, lengths)
    q = _randn(g, b, 4, 1, d)
    starts = _i32([x * members for x in range(groups + 1)])
    o, lse = wise.prefix_attention(q, cache, _i32([prefix] * groups), group_starts=starts, out_dtype=torch.float32)
    ro, rl = wise.tree_attention(q, cache, out_dtype=torch.float32)
    wise.check_device()
    # sum a |v| below 4; both sides within 2 * 2^-8 + 2^-10 of it (weights rounded to bf16, scores' sums)
    assert float((o - ro).abs().max()) <= 2 * (2.0 ** -7 + 2.0 ** -10) * 4.0 and float((lse - rl).abs().max()) <= 2.0 ** -14
    # with the groups' size known, by the kernel for few rows
    o, lse = wise.prefix_attention(q, cache, _i32([prefix] * groups), group_starts=starts, max_members=members, out_dtype=torch.float32)
    wise.check_device()
    assert float((o - ro).abs().max()) <= 2 * (2.0 ** -7 + 2.0 ** -10) * 4.0 and float((lse - rl).abs().max()) <= 2.0 ** -14


@pytest.mark.parametrize("most", [1, 2, 3, 6, 40])
def test_groups_larger_than_said_share_nothing(most):
    """Sizes of groups that are not what the caller said are flagged; results stay."""
    rng = np.random.default_rng(33)
    starts, prefixes = [0, 2, 3, 6], [256, 300, 390]
    lengths = [260, 270, 300, 400, 390, 444]
    cache, table = _shared_cache(rng, starts, prefixes, lengths, [3] * 6, 2, 96, 32)
    q = _bf16(rng.standard_normal((6, 12, 3, 96)))
    sees = _mask(rng, 6, 3, "run")[0]
    got = wise.prefix_attention(q, cache, _i32(prefixes), group_starts=_i32(starts), max_members=most, out_dtype=torch.float32)
    assert wise.device_status() == (wise._lib.WISE_ERR_BAD_CACHE if most < 3 else 0)
    _check(q, cache, table, sees, lengths, [3] * 6, got, torch.float32)


def test_rows_past_the_page_table_are_empty():
    """Where new tokens do not fit the table, rows behind those that do see
    nothing, as in the attention without sharing."""
    rng = np.random.default_rng(31)
    lengths = [142, 140]
    cache, table = _shared_cache(rng, [0, 2], [128], lengths, [2, 4], 2, 64, 16)
    full = wise.PagedCache(cache.k_pages, cache.v_pages, cache.page_table[:, :9].contiguous(), cache.lengths)  # 144 tokens
    q = _bf16(rng.standard_normal((2, 4, 4, 64)))
    o, lse = wise.prefix_attention(q, full, _i32([128]), out_dtype=torch.float32)
    assert wise.device_status() == wise._lib.WISE_ERR_BAD_CACHE
    ro, rl = wise.tree_attention(q, full, out_dtype=torch.float32)
    assert wise.device_status() == wise._lib.WISE_ERR_BAD_CACHE
    assert torch.equal(torch.isneginf(lse), torch.isneginf(rl)) and bool(torch.isneginf(lse[0, :, 2:]).all())
    assert torch.all(o[0, :, 2:] == 0) and not torch.isneginf(lse[0, :, :2]).any() and not torch.isneginf(lse[1]).any()


class _Server:
    """A small serving loop over one cache: append with norms, shared-prefix
    attention, weights, acceptance; eviction at the end."""

    def __init__(self, seed, b=3, hk=2, h=8, d=64, page=32, prompt=300, steps=6):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.b, self.steps, self.prompt = b, steps, prompt
        cols = (prompt + 3 * steps + page) // page + 1
        whole = prompt // page
        kept = (100 + page - 1) // page
        pages = whole + b * (cols - whole) + b * kept
        self.k, self.v = (_randn(g, pages, hk, page, d) for _ in range(2))
        t = torch.full((b, cols), -1, dtype=torch.int32, device="cuda")
        t[:, :whole] = torch.arange(whole, device="cuda")
        t[:, whole:] = whole + torch.arange(b * (cols - whole), device="cuda").reshape(b, -1)
        self.table = t
        self.to = (pages - b * kept + torch.arange(b * kept, device="cuda")).to(torch.int32).reshape(b, kept)
        left = prompt % page
        for p in (self.k, self.v):
            p[t[1:, whole].long(), :, :left] = p[int(t[0, whole]), :, :left]
        self.x = [[_randn(g, b, m, 3, d) for m in (hk, hk, h)] for _ in range(steps)]
        self.news = [_i32([3 - (s + i) % 3 for i in range(b)]) for s in range(steps)]
        self.rope = wise.rope_frequencies(d, sections=(10, 11, d // 2 - 21))
        self.pos = [torch.randint(0, 400, (3, b, 3), generator=g, device="cuda").to(torch.int32) for _ in range(steps)]
        self.qn, self.kn = (torch.rand((m, d), generator=g, device="cuda") + 0.5 for m in (h, hk))
        self.pre = _i32([prompt])
        self.k0, self.v0 = self.k.clone(), self.v.clone()
        self.weights = torch.zeros((b, hk, cols * page), device="cuda")
        self.start = torch.full((b,), prompt, dtype=torch.int32, device="cuda")

    def reset(self):
        self.k.copy_(self.k0)
        self.v.copy_(self.v0)
        self.weights.zero_()

    def run(self, stream=None):
        out, lengths = [], self.start
        for s in range(self.steps):
            cache = wise.PagedCache(self.k, self.v, self.table, lengths)
            x = self.x[s]
            q = wise.cache_append(cache, x[0], x[1], q=x[2], new_len=self.news[s], positions=self.pos[s], rope=self.rope,
                                  q_norm=self.qn, k_norm=self.kn, stream=stream)
            o, lse = wise.prefix_attention(q, cache, self.pre, new_len=self.news[s], stream=stream)
            wise.cache_weights(q, cache, lse, self.weights, new_len=self.news[s], stream=stream)
            lengths = wise.cache_accept(cache, self.news[s], stream=stream)
            out += [q, o, lse, lengths]
        small, kept = wise.cache_evict(wise.PagedCache(self.k, self.v, self.table, lengths), self.weights, 100, self.to, recent=9,
                                       sink=3, stream=stream)
        dense = wise.norm_rotate(self.x[0][2], self.x[0][0], q_norm=self.qn, k_norm=self.kn, positions=self.pos[0], rope=self.rope,
                                 stream=stream)
        return out + [small.lengths, kept, *dense]

    def state(self):
        return [self.k, self.v, self.weights]


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b)) and len(a) == len(b)


def _reference(server):
    server.reset()
    out = [x.clone() for x in server.run()]
    torch.cuda.synchronize()
    wise.check_device()
    return out, [x.clone() for x in server.state()]


def test_calls_one_after_the_other():
    """The loop without a pause, twenty times, gives the bits of its first run:
    no launch reads what the one before it has not finished."""
    s = _Server(1)
    want, state = _reference(s)
    for _ in range(20):
        s.reset()
        got = s.run()
        assert _same(got, want) and _same(s.state(), state)
    wise.check_device()


def test_inputs_rewritten_in_place_between_calls():
    """Lengths, page table, groups, new tokens' counts, queries and pages that are
    written again, at the same addresses, right before each call: every call sees
    what was written last."""
    g = torch.Generator(device="cuda").manual_seed(13)
    b, h, hk, d, page, n, cols, pages = 6, 8, 2, 64, 16, 2, 40, 120
    k, v = (_randn(g, 3, pages, hk, page, d) for _ in range(2))
    kinds = []
    for i in range(5):
        prefix = [256, 128, 400, 384, 130][i]
        table = torch.randperm(pages, generator=g, device="cuda")[:cols].to(torch.int32).expand(b, cols).clone()
        own = torch.randperm(pages, generator=g, device="cuda")[:b * 10].to(torch.int32).reshape(b, 10)
        table[:, prefix // page:prefix // page + 10] = own
        table[:, prefix // page] = table[0, prefix // page]
        lengths = prefix + torch.randint(0, 100, (b,), generator=g, device="cuda").to(torch.int32)
        starts = _i32([[0, 6], [1, 5], [0, 3], [2, 6], [0, 6]][i])
        kinds.append(dict(lengths=lengths, table=table, starts=starts, pre=_i32([prefix]), q=_randn(g, b, h, n, d),
                          news=torch.randint(0, n + 1, (b,), generator=g, device="cuda").to(torch.int32), k=k[i % 3], v=v[(i + 1) % 3]))
    wants = []
    for x in kinds:
        cache = wise.PagedCache(x["k"].contiguous(), x["v"].contiguous(), x["table"], x["lengths"])
        o, lse = wise.prefix_attention(x["q"], cache, x["pre"], group_starts=x["starts"], new_len=x["news"])
        w = wise.cache_weights(x["q"], cache, lse, torch.zeros((b, hk, 700), device="cuda"), new_len=x["news"])
        torch.cuda.synchronize()
        wants.append((o, lse, w))
    wise.check_device()
    now = {key: torch.empty_like(t) for key, t in kinds[0].items()}
    cache = wise.PagedCache(now["k"], now["v"], now["table"], now["lengths"])
    o, lse, w = (torch.empty_like(t) for t in wants[0])
    order = np.random.default_rng(14).integers(0, 5, 150)
    got = []
    for i in order:
        for key, t in kinds[i].items():
            now[key].copy_(t)
        w.zero_()
        wise.prefix_attention(now["q"], cache, now["pre"], group_starts=now["starts"], new_len=now["news"], out=o, lse=lse)
        wise.cache_weights(now["q"], cache, lse, w, new_len=now["news"])
        got.append((o.clone(), lse.clone(), w.clone()))
    wise.check_device()
    for i, x in zip(order, got):
        assert _same(x, wants[i])


def test_two_graphs_in_turn():
    a, b = _Server(2), _Server(3, b=4, hk=1, h=4, d=128, page=16, prompt=200, steps=3)
    wants = [_reference(x) for x in (a, b)]
    graphs, outs = [], []
    for x in (a, b):
        x.reset()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(x.run())
        graphs.append(g)
    for _ in range(3):
        for x in (a, b):
            x.reset()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for x, o, (want, state) in zip((a, b), outs, wants):
            assert _same(o, want) and _same(x.state(), state)
    wise.check_device()


def test_streams():
    """Two loops at the same time on given streams, and one on the current one."""
    servers = [_Server(4), _Server(5), _Server(6, h=2, d=96)]
    wants = [_reference(x) for x in servers]
    streams = [torch.cuda.Stream(), torch.cuda.Stream(), None]
    for _ in range(5):
        for x in servers:
            x.reset()
        for st in streams[:2]:
            st.wait_stream(torch.cuda.current_stream())
        got = [x.run(st) for x, st in zip(servers, streams)]
        torch.cuda.synchronize()
        for x, o, (want, state) in zip(servers, got, wants):
            assert _same(o, want) and _same(x.state(), state)
    wise.check_device()


FIRST = """
import sys
sys.path.insert(0, {root!r})
import torch
import block_sparse_attention_causal_gb300 as wise
from tests.test_gpu_more_forms import _Server
s = _Server(7)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = s.run()
g.replay()
torch.cuda.synchronize()
got, state = [x.clone() for x in out], [x.clone() for x in s.state()]
s.reset()
want = s.run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(torch.equal(a, b) for a, b in zip(state, s.state()))
wise.check_device()
print("same")
"""


def test_a_process_s_first_calls_recorded_into_a_graph():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=root)], capture_output=True, text=True, timeout=300, cwd=root)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr


def test_given_buffers():
    s = _Server(8)
    cache = wise.PagedCache(s.k, s.v, s.table, s.start)
    q = s.x[0][2]
    want = wise.prefix_attention(q, cache, s.pre, scale=0.3)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    desc = wise._check_cache(cache)[0]
    ws = torch.full((wise._lib.load().wise_attn_prefix_workspace(desc, 8, 3, 1) + 5,), 255, dtype=torch.uint8, device="cuda")
    got = wise.prefix_attention(q, cache, s.pre, scale=0.3, out=out, lse=lse, workspace=ws)
    assert got[0] is out and got[1] is lse and _same(got, want)
    assert wise.prefix_attention(q, cache, s.pre, scale=0.3, want_lse=False)[1] is None
    lens, w = torch.empty(3, dtype=torch.int32, device="cuda"), torch.empty((3, 2, 50), device="cuda")
    s.weights.uniform_()
    ws = torch.empty(3 * 2 * 40 * 4, dtype=torch.uint8, device="cuda")
    small, kept = wise.cache_evict(cache, s.weights, 40, s.to, recent=3, new_lengths=lens, weights_out=w, workspace=ws)
    assert small.lengths is lens and kept is w
    again, kept2 = wise.cache_evict(cache, s.weights, 40, s.to, recent=3)
    assert torch.equal(lens, again.lengths) and torch.equal(w[..., :40], kept2[..., :40]) and not w[..., 40:].any()
    wise.check_device()
    for bad in (lambda: wise.prefix_attention(q, cache, s.pre, workspace=ws), lambda: wise.prefix_attention(q, cache, s.pre, out=out[:1]),
                lambda: wise.prefix_attention(q[:, :3], cache, s.pre), lambda: wise.prefix_attention(q, cache, _i32([300, 300])),
                lambda: wise.prefix_attention(q, cache, s.pre.long()), lambda: wise.prefix_attention(q, cache, s.pre, group_starts=_i32([0])),
                lambda: wise.prefix_attention(q, cache, s.pre, out_dtype=torch.float16), lambda: wise.prefix_attention(q, cache, s.pre, max_members=-1),
                lambda: wise.cache_weights(q, cache, lse[:, :2], s.weights), lambda: wise.cache_weights(q, cache, lse, s.weights[0]),
                lambda: wise.cache_weights(q, cache, lse, s.weights.double()), lambda: wise.cache_weights(q, cache, lse.half(), s.weights),
                lambda: wise.cache_weights(q, cache, lse, s.weights[..., ::2]),
                lambda: wise.cache_evict(cache, s.weights, 40.0, s.to), lambda: wise.cache_evict(cache, s.weights, 40, s.to[0]),
                lambda: wise.cache_evict(cache, s.weights, -1, s.to), lambda: wise.cache_evict(cache, s.weights, 40, s.to, recent=1 << 31),
                lambda: wise.cache_evict(cache, s.weights, 40, s.to, workspace=ws[:8]),
                lambda: wise.cache_evict(cache, s.weights, 40, s.to, new_lengths=lens.long()),
                lambda: wise.cache_append(cache, s.x[0][0], s.x[0][1], q_norm=s.qn, rope=s.rope),
                lambda: wise.cache_append(cache, s.x[0][0], s.x[0][1], rope=s.rope),  # axes, but no positions
                lambda: wise.cache_append(cache, s.x[0][0], s.x[0][1], rope=s.rope, positions=s.pos[0][0].contiguous()),
                lambda: wise.cache_append(cache, s.x[0][0], s.x[0][1], k_norm=s.qn),
                lambda: wise.cache_append(cache, s.x[0][0], s.x[0][1], q=q, k_norm=s.kn, q_norm=s.qn.to(torch.bfloat16)),
                lambda: wise.norm_rotate(q, k_norm=s.kn), lambda: wise.norm_rotate(q, s.x[0][0][:, :, :2]),
                lambda: wise.norm_rotate(q.float()), lambda: wise.norm_rotate(q, q_norm=s.qn, norm_eps=0.0)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: wise.cache_evict(cache, s.weights, 40, s.to, recent=41), lambda: wise.cache_evict(cache, s.weights, 0, s.to),
                lambda: wise.cache_evict(cache, s.weights, 129, s.to), lambda: wise.cache_evict(cache, s.weights, 40, s.to, weights_out=w[..., :39].contiguous()),
                lambda: wise.cache_evict(cache, s.weights, 40, s.to, new_lengths=cache.lengths),
                lambda: wise.prefix_attention(q, cache, s.pre, out=q), lambda: wise.norm_rotate(q, q_out=q)):
        with pytest.raises(wise.WiseError):
            bad()
    wise.check_device()


def test_pools_past_32_bits():
    """Pages whose elements lie past 2^32, against the same pages in a small pool."""
    g = torch.Generator(device="cuda").manual_seed(11)
    hk, page, d, b, h = 1, 128, 128, 2, 4
    far = (1 << 32) // (hk * page * d) + 3
    big = [torch.zeros((far + 12, hk, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    small = [torch.zeros((12, hk, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    rows = _randn(g, 12, hk, page, d), _randn(g, 12, hk, page, d)
    table = _i32([[0, 1, 2, -1], [0, 1, 3, -1]])
    to = _i32([[8, 9], [10, 11]])
    x = [_randn(g, b, m, 2, d) for m in (hk, hk, h)]
    rope, kn, qn = wise.rope_frequencies(d), torch.rand(d, generator=g, device="cuda") + 0.5, torch.rand(d, generator=g, device="cuda") + 0.5
    out = []
    for pools, at in ((small, 0), (big, far)):
        for p, r in zip(pools, rows):
            p[at:at + 12] = r
        cache = wise.PagedCache(pools[0], pools[1], torch.where(table < 0, table, table + at).to(torch.int32), _i32([300, 290]))
        q = wise.cache_append(cache, x[0], x[1], q=x[2], rope=rope, q_norm=qn, k_norm=kn)
        o, lse = wise.prefix_attention(q, cache, _i32([256]))
        w = wise.cache_weights(q, cache, lse, torch.zeros((b, hk, 400), device="cuda"))
        kept, w2 = wise.cache_evict(cache, w, 150, (to + at).to(torch.int32), recent=10)
        wise.check_device()
        out.append([q, o, lse, w, w2, kept.lengths] + [p[at:at + 12].clone() for p in pools])
    assert _same(*out)


def test_dense_rows_past_32_bits():
    """2^31 elements and more, laid out token by token."""
    g = torch.Generator(device="cuda").manual_seed(12)
    h, n, d = 17, 1 << 20, 128
    q = torch.empty((1, n, h, d), dtype=torch.bfloat16, device="cuda")
    for i in range(0, n, 1 << 17):
        q[:, i:i + (1 << 17)] = _randn(g, 1, 1 << 17, h, d)
    q = q.transpose(1, 2)
    w, rope = torch.rand(d, generator=g, device="cuda") + 0.5, wise.rope_frequencies(d)
    out, _ = wise.norm_rotate(q, q_norm=w, rope=rope)
    for i in (0, 12345, n - 40):
        pos = torch.arange(i, i + 40, dtype=torch.int32, device="cuda")[None].contiguous()
        few, _ = wise.norm_rotate(q[:, :, i:i + 40], q_norm=w, rope=rope, positions=pos)
        assert torch.equal(out[:, :, i:i + 40], few)
    wise.check_device()
