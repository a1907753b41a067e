"""Refusals of norms with rotation, shared-prefix attention, gathered weights and
eviction, on the host before any launch."""
import numpy as np
import pytest
import torch

import block_sparse_attention_causal_gb300 as wise
from block_sparse_attention_causal_gb300 import _lib
from oracle import cache_oracle as C

E = _lib
MB = 1 << 20


def _cache(batch=2, kv_heads=2, head_dim=64, page=16, max_pages=4, n_pages=8, kp=1 * MB, vp=2 * MB, table=3 * MB, lengths=4 * MB):
    return _lib.PagedCacheDesc(batch, kv_heads, head_dim, page, max_pages, 0, n_pages, kp, vp, table, lengths)


def _rows(data=16 * MB, strides=(64, 64, 64)):
    r = _lib.Rows(data)
    r.stride[:] = strides
    return r


def _rope(steps=20 * MB, axes=None, rotary=64, n_axes=1, flags=0):
    return _lib.RopeDesc(steps, axes, rotary, n_axes, flags, 0)


def _norm(q=21 * MB, k=22 * MB, q_step=0, k_step=0, kind=E.WISE_F32, eps=1e-6):
    return _lib.HeadNorm(q, k, q_step, k_step, kind, eps)


INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = (E.WISE_ERR_INVALID_ARGUMENT, E.WISE_ERR_UNSUPPORTED, E.WISE_ERR_ALIGNMENT,
                                             E.WISE_ERR_WORKSPACE)

BAD_CACHES = [
    (dict(batch=0), INVALID), (dict(kv_heads=0), INVALID), (dict(max_pages=0), INVALID), (dict(n_pages=0), INVALID),
    (dict(batch=65536), UNSUPPORTED), (dict(head_dim=80), UNSUPPORTED), (dict(page=8), UNSUPPORTED),
    (dict(page=128, max_pages=(1 << 23) + 1), UNSUPPORTED), (dict(kp=None), INVALID), (dict(vp=None), INVALID),
    (dict(table=None), INVALID), (dict(lengths=None), INVALID), (dict(kp=8), ALIGNMENT), (dict(vp=24), ALIGNMENT),
    (dict(table=6), ALIGNMENT), (dict(lengths=2), ALIGNMENT),
]


@pytest.mark.parametrize("bad,status", BAD_CACHES, ids=lambda x: str(x))
def test_bad_cache_descriptors(lib, bad, status):
    c = _cache(**bad)
    assert lib.wise_cache_append_norm(c, 1, _rows(), _rows(), 0, None, None, None, None, None, None, None) == status
    assert lib.wise_attn_prefix(c, 2, 1, _rows(), 1, 0, None, 16, None, None, 0.0, 0, 16, None, 16, 1 << 30, None) == status
    assert lib.wise_cache_weights(c, 2, 1, _rows(), 16, None, None, 0.0, 64 * MB, 8, None) == status
    assert lib.wise_cache_evict(c, 16, 8, 4, 0, 0, 16, 1, 64 * MB, 65 * MB, 8, 66 * MB, 1 << 20, None) == status


NORM_REFUSALS = [
    (dict(rope=dict(rotary=-16)), INVALID), (dict(rope=dict(rotary=8)), INVALID), (dict(rope=dict(rotary=80)), INVALID),
    (dict(rope=dict(steps=None)), INVALID), (dict(rope=dict(steps=20 * MB + 4)), ALIGNMENT), (dict(rope=dict(flags=2)), INVALID),
    (dict(rope=dict(n_axes=0)), INVALID), (dict(rope=dict(n_axes=2)), INVALID),  # more axes than one without naming them
    (dict(rope=dict(axes=23 * MB, n_axes=2), positions=None), INVALID),
    (dict(rope=dict(axes=23 * MB + 2, n_axes=2)), ALIGNMENT),
    (dict(norm=dict(eps=0.0)), INVALID), (dict(norm=dict(eps=-1.0)), INVALID), (dict(norm=dict(eps=float("nan"))), INVALID),
    (dict(norm=dict(eps=float("inf"))), INVALID), (dict(norm=dict(kind=2)), INVALID), (dict(norm=dict(q_step=-8)), INVALID),
    (dict(norm=dict(q=21 * MB + 8)), ALIGNMENT), (dict(norm=dict(k=22 * MB + 4)), ALIGNMENT), (dict(norm=dict(k_step=4)), ALIGNMENT),
    (dict(norm=dict(q_step=1 << 62)), UNSUPPORTED),
    (dict(positions=24 * MB + 2), ALIGNMENT), (dict(q=_rows(None)), INVALID), (dict(q=_rows(8)), ALIGNMENT),
    (dict(k=_rows(strides=(64, 4, 64))), ALIGNMENT), (dict(k=_rows(strides=(64, -64, 64))), INVALID),
    (dict(q_out=None), INVALID), (dict(q_out=8), ALIGNMENT), (dict(heads=0), INVALID), (dict(heads=1 << 18), UNSUPPORTED),
    (dict(n=0), INVALID), (dict(n=1 << 30), UNSUPPORTED),
    # results over what is read
    (dict(q_out=20 * MB + 16), INVALID), (dict(q_out=21 * MB), INVALID), (dict(q_out=22 * MB + 128), INVALID),
    (dict(q_out=24 * MB), INVALID), (dict(rope=dict(axes=23 * MB, n_axes=1), q_out=23 * MB + 64), INVALID),
    (dict(q_out=16 * MB + 256), INVALID),
    (dict(norm=dict(q_step=64), q_out=21 * MB + 64 * 4), INVALID),  # the second head's weights
]


@pytest.mark.parametrize("bad,status", NORM_REFUSALS, ids=lambda x: str(x) if isinstance(x, int) else "-".join(x))
def test_norm_arguments(lib, bad, status):
    args = dict(dict(n=3, heads=2, q=_rows(), k=_rows(), q_out=32 * MB, positions=24 * MB), **{k: v for k, v in bad.items() if k not in ("rope", "norm")})
    rope, norm = _rope(**bad.get("rope", {})), _norm(**bad.get("norm", {}))
    got = lib.wise_cache_append_norm(_cache(), args["n"], args["k"], _rows(), args["heads"], args["q"], args["q_out"], None,
                                     args["positions"], rope, norm, None)
    assert got == status
    got = lib.wise_norm_rotate(2, args["n"], 64, args["heads"], args["q"], args["q_out"], 2, args["k"], 40 * MB, args["positions"],
                               rope, norm, None)
    assert got == status


def test_append_with_norms_refuses_more(lib):
    def call(c=None, v=None, new_len=None, q_out=32 * MB):
        return lib.wise_cache_append_norm(c or _cache(), 3, _rows(), v or _rows(), 2, _rows(), q_out, new_len, None, _rope(), _norm(), None)
    assert call(v=_rows(None)) == INVALID
    assert call(new_len=2) == ALIGNMENT
    assert call(new_len=32 * MB + 16) == INVALID
    assert call(c=_cache(vp=1 * MB + 64)) == INVALID  # one pool for keys and values
    for over in (1 * MB, 2 * MB + 4096, 3 * MB, 4 * MB):
        assert call(q_out=over) == INVALID


def test_norm_rotate_refuses_more(lib):
    def call(batch=2, d=64, kv=2, k=_rows(), k_out=40 * MB, q_out=32 * MB):
        return lib.wise_norm_rotate(batch, 3, d, 2, _rows(), q_out, kv, k, k_out, None, _rope(rotary=0), _norm(), None)
    assert call(batch=0) == INVALID and call(d=32) == UNSUPPORTED and call(kv=0) == INVALID and call(k_out=None) == INVALID
    assert call(k_out=8) == ALIGNMENT
    size = 2 * 2 * 3 * 64 * 2
    for at in (32 * MB, 32 * MB + size - 16, 32 * MB - size + 16, 16 * MB, 21 * MB, 22 * MB):
        assert call(k_out=at) == INVALID, hex(at)


def test_prefix_arguments(lib):
    ws = lib.wise_attn_prefix_workspace(_cache(), 4, 3, 1)
    assert ws > lib.wise_attn_tree_workspace(_cache(), 4, 3)

    def call(c=None, heads=4, n=3, q=None, groups=1, members=0, starts=None, pre=48 * MB, new_len=None, mask=None, scale=0.0, dtype=0,
             o=32 * MB, lse=None, w=64 * MB, wb=ws):
        return lib.wise_attn_prefix(c or _cache(), heads, n, q or _rows(), groups, members, starts, pre, new_len, mask, scale, dtype, o, lse,
                                    w, wb, None)
    assert call(heads=3) == INVALID and call(heads=0) == INVALID and call(n=0) == INVALID and call(n=129) == UNSUPPORTED
    assert call(groups=0) == INVALID and call(groups=3) == INVALID  # more groups than sequences
    assert call(groups=2, wb=1 << 30) == INVALID                    # two groups without their starts
    assert call(pre=None) == INVALID and call(pre=2) == ALIGNMENT and call(starts=50 * MB + 1) == ALIGNMENT
    assert call(members=-1) == INVALID and call(dtype=2) == INVALID and call(scale=-1.0) == INVALID and call(scale=float("nan")) == INVALID
    assert call(o=None) == INVALID and call(o=8) == ALIGNMENT and call(lse=2) == ALIGNMENT and call(mask=2) == ALIGNMENT
    assert call(new_len=2) == ALIGNMENT and call(q=_rows(strides=(64, 64, 12))) == ALIGNMENT
    assert call(w=None) == WORKSPACE and call(wb=ws - 1) == WORKSPACE and call(w=64 * MB + 8) == ALIGNMENT
    # results and workspace over inputs and each other
    for over in (1 * MB, 2 * MB, 3 * MB, 4 * MB, 16 * MB, 48 * MB, 64 * MB):
        assert call(o=over) == INVALID, hex(over)
        assert call(lse=over) == INVALID, hex(over)
    assert call(w=48 * MB - 64) == INVALID and call(starts=32 * MB) == INVALID and call(new_len=32 * MB) == INVALID
    assert call(mask=64 * MB + 256) == INVALID and call(lse=32 * MB + 32) == INVALID
    for bad in (dict(c=_cache(head_dim=32)), dict(heads=5), dict(n=0), dict(n=129), dict(groups=0), dict(groups=3)):
        assert lib.wise_attn_prefix_workspace(bad.get("c", _cache()), bad.get("heads", 4), bad.get("n", 3), bad.get("groups", 1)) == 0
    assert lib.wise_attn_prefix_workspace(_cache(kp=None, vp=None, table=None, lengths=None), 4, 3, 1) == ws


def test_weights_arguments(lib):
    def call(c=None, heads=4, n=3, q=None, lse=48 * MB, new_len=None, mask=None, scale=0.0, w=32 * MB, width=70):
        return lib.wise_cache_weights(c or _cache(), heads, n, q or _rows(), lse, new_len, mask, scale, w, width, None)
    assert call(heads=3) == INVALID and call(n=0) == INVALID and call(n=129) == UNSUPPORTED
    assert call(lse=None) == INVALID and call(w=None) == INVALID and call(width=0) == INVALID and call(scale=-1.0) == INVALID
    assert call(width=1 << 62) == UNSUPPORTED
    assert call(lse=2) == ALIGNMENT and call(w=2) == ALIGNMENT and call(new_len=2) == ALIGNMENT and call(mask=2) == ALIGNMENT
    assert call(q=_rows(8)) == ALIGNMENT and call(q=_rows(None)) == INVALID
    for over in (1 * MB, 2 * MB, 3 * MB, 4 * MB, 16 * MB, 48 * MB):
        assert call(w=over) == INVALID, hex(over)
    assert call(new_len=32 * MB + 4) == INVALID and call(mask=32 * MB + 8) == INVALID


def test_evict_arguments(lib):
    ws = lib.wise_cache_evict_workspace(_cache(), 20)
    assert ws == 2 * 2 * 20 * 4 and lib.wise_cache_evict_workspace(_cache(), 0) == 0
    assert lib.wise_cache_evict_workspace(_cache(page=8), 20) == 0

    def call(c=None, w=16 * MB, width=64, budget=20, recent=3, sink=2, to=20 * MB, pages=2, lens=24 * MB, wo=32 * MB, wide=32,
             work=40 * MB, wb=ws):
        return lib.wise_cache_evict(c or _cache(), w, width, budget, recent, sink, to, pages, lens, wo, wide, work, wb, None)
    for bad in (dict(w=None), dict(to=None), dict(lens=None), dict(wo=None), dict(width=0), dict(pages=0), dict(budget=0),
                dict(recent=-1), dict(sink=-1), dict(recent=19), dict(sink=18), dict(wide=19), dict(pages=1)):
        assert call(**bad) == INVALID, bad
    assert call(recent=2 ** 31 - 1, sink=2 ** 31 - 1) == INVALID
    assert call(width=1 << 62) == UNSUPPORTED and call(wide=1 << 62) == UNSUPPORTED and call(pages=1 << 27) == UNSUPPORTED
    for name in ("w", "to", "lens", "wo"):
        assert call(**{name: 16 * MB + 2}) == ALIGNMENT, name
    assert call(work=None) == WORKSPACE and call(wb=ws - 1) == WORKSPACE and call(work=40 * MB + 8) == ALIGNMENT
    assert call(c=_cache(vp=1 * MB)) == INVALID
    for over in (1 * MB, 2 * MB, 3 * MB, 4 * MB, 16 * MB, 20 * MB):  # pools, table, lengths, weights, the new table
        for name in ("lens", "wo", "work"):
            assert call(**{name: over}) == INVALID, (name, hex(over))
    assert call(lens=32 * MB + 64) == INVALID and call(work=32 * MB + 64) == INVALID and call(work=24 * MB) == INVALID
    # what the call reads must not lie in the pools that it writes
    assert call(w=1 * MB + 64) == INVALID and call(to=2 * MB + 64) == INVALID


def test_python_refusals():
    """Without a device: what is refused before one is asked."""
    rope = wise.rope_frequencies(64, device="cpu")
    ok = torch.zeros((2, 2, 3, 64), dtype=torch.bfloat16)
    for call in (lambda: wise.norm_rotate(ok[0]), lambda: wise.norm_rotate(ok), lambda: wise.norm_rotate(None),
                 lambda: wise._check_norms(torch.ones(64, dtype=torch.float16), 2, None, 2, 64, 1e-6, -1),
                 lambda: wise._check_norms(None, 2, "w", 2, 64, 1e-6, -1),
                 lambda: wise._check_norms(torch.ones(64), 2, None, 2, 64, 1e-6, -1),  # not on a device
                 lambda: wise._check_positions("rope", None, 2, 3, -1),
                 lambda: wise.rope_frequencies(64, sections=(16, 15), device="cpu"),
                 lambda: wise.rope_frequencies(64, sections=(), device="cpu")):
        with pytest.raises(ValueError):
            call()
    rope.axes = torch.zeros(32, dtype=torch.int32)
    with pytest.raises(ValueError):
        wise._check_positions(rope, None, 2, 3, -1)
    assert wise._check_norms(None, 2, None, 2, 64, 0.0, -1) is None
    assert wise.rope_frequencies(64, sections=(20, 0, 12), device="cpu").axes.tolist() == [0] * 20 + [2] * 12


def test_oracle_norm_rotation_keeps_lengths():
    """Unit weights, no eps: rows come out with length sqrt(d); rotation by one
    axis named for every pair is rotation without axes."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal(96)
    freq = [100.0 ** (-i / 24) for i in range(24)]
    y, _ = C.norm_rotate(x, 17, freq, True, np.ones(96), 0.0)
    assert abs(np.linalg.norm(y) - np.sqrt(96)) < 1e-12
    z, _ = C.norm_rotate(x, [3, 17], freq, True, np.ones(96), 0.0, axes=[1] * 24)
    assert np.array_equal(y, z)
    assert np.allclose(C.norm_rotate(x, 5, freq, False)[0], C.rotate(x, 5, freq, False), atol=0)


def test_oracle_weights_are_softmax_columns():
    rng = np.random.default_rng(1)
    k = rng.standard_normal((4, 1, 16, 64))
    q = rng.standard_normal((1, 2, 3, 64))
    table, lengths = [[0, 1, 2, 3]], [20]
    sees = np.tril(np.ones((1, 3, 3), bool))
    _, lse, _, _ = C.tree_attention(q, k, k, table, lengths, sees)
    w, _ = C.gather_weights(q, k, table, lengths, sees, lse, np.full((1, 1, 30), 0.5))
    assert np.allclose(w[0, 0, :23].sum(), 0.5 * 20 + 6) and np.all(w[0, 0, 23:] == 0.5)


def test_oracle_kept_tokens():
    w = [0.0, 5.0, np.nan, 5.0, 1.0, -1.0, 9.0, 0.0]
    assert C.kept_tokens(w, 8, 3, 1, 0) == [1, 6, 7]
    assert C.kept_tokens(w, 8, 3, 0, 1) == [0, 1, 6]
    assert C.kept_tokens(w, 8, 7, 0, 0) == [0, 1, 3, 4, 5, 6, 7]  # NaN goes first
    assert C.kept_tokens(w, 8, 8, 2, 2) == list(range(8))


def test_prefix_workspace_grows_with_the_batch_alone(lib):
    """Two rows of fp32 results a query row, records of the units, partial results
    of the blocks (304 of 256 rows and statistics): no product of groups and rows."""
    for batch, groups in ((64, 1), (64, 64), (8192, 1), (8192, 8192), (65535, 65535)):
        c = _cache(batch=batch, kv_heads=8, head_dim=128, page=64, kp=None, vp=None, table=None, lengths=None)
        rows = batch * 32
        parts = 304 * (256 * 128 + 2 * 256) * 4
        most = rows * 2 * (128 + 1) * 4 + 2 * parts + (batch * 8 + (batch * 4 // 256 + groups + 1) * 8) * 32 + (3 * groups + 3 * batch + 3) * 4 + 8192
        assert 0 < lib.wise_attn_prefix_workspace(c, 32, 1, groups) <= most
