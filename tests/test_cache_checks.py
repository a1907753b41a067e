"""Refusals of the paged-cache calls, on the host before any launch."""
import ctypes

import pytest
import torch

import block_sparse_attention_causal_gb300 as wise
from block_sparse_attention_causal_gb300 import _lib

E = _lib


def _cache(batch=2, kv_heads=2, head_dim=64, page=16, max_pages=4, n_pages=8, kp=16, vp=16, table=16, lengths=1 << 20):
    return _lib.PagedCacheDesc(batch, kv_heads, head_dim, page, max_pages, 0, n_pages, kp, vp, table, lengths)


def _rows(data=16, strides=(64, 64, 64)):
    r = _lib.Rows(data)
    r.stride[:] = strides
    return r


BAD_CACHES = [
    (dict(batch=0), E.WISE_ERR_INVALID_ARGUMENT), (dict(kv_heads=0), E.WISE_ERR_INVALID_ARGUMENT),
    (dict(max_pages=0), E.WISE_ERR_INVALID_ARGUMENT), (dict(n_pages=0), E.WISE_ERR_INVALID_ARGUMENT),
    (dict(batch=65536), E.WISE_ERR_UNSUPPORTED), (dict(head_dim=80), E.WISE_ERR_UNSUPPORTED),
    (dict(page=8), E.WISE_ERR_UNSUPPORTED), (dict(page=48), E.WISE_ERR_UNSUPPORTED),
    (dict(page=128, max_pages=(1 << 23) + 1), E.WISE_ERR_UNSUPPORTED), (dict(n_pages=1 << 31), E.WISE_ERR_UNSUPPORTED),
    (dict(kp=None), E.WISE_ERR_INVALID_ARGUMENT), (dict(vp=None), E.WISE_ERR_INVALID_ARGUMENT),
    (dict(table=None), E.WISE_ERR_INVALID_ARGUMENT), (dict(lengths=None), E.WISE_ERR_INVALID_ARGUMENT),
    (dict(kp=8), E.WISE_ERR_ALIGNMENT), (dict(vp=24), E.WISE_ERR_ALIGNMENT), (dict(table=6), E.WISE_ERR_ALIGNMENT),
    (dict(lengths=2), E.WISE_ERR_ALIGNMENT),
]


@pytest.mark.parametrize("bad,status", BAD_CACHES, ids=lambda x: str(x))
def test_bad_cache_descriptors(lib, bad, status):
    c = _cache(**bad)
    ws = 1 << 30
    assert lib.wise_cache_append(c, 1, _rows(), _rows(), 0, None, None, None, None, None, 0, 0, None) == status
    assert lib.wise_attn_tree(c, 2, 1, _rows(), None, None, 0.0, 0, 16, None, 16, ws, None) == status
    assert lib.wise_cache_accept(c, 1, None, 16, 64, None) == status


def test_append_arguments(lib):
    def call(c=None, n=3, k=None, v=None, heads=2, q=None, q_out=None, new_len=None, positions=None, rope=16, rotary=64,
             flags=0):
        return lib.wise_cache_append(c or _cache(), n, k or _rows(), v or _rows(), heads, q, q_out, new_len, positions,
                                     rope, rotary, flags, None)
    assert call(n=0) == E.WISE_ERR_INVALID_ARGUMENT
    assert call(q=_rows()) == E.WISE_ERR_INVALID_ARGUMENT              # no q_out
    assert call(q=_rows(), q_out=16, heads=0) == E.WISE_ERR_INVALID_ARGUMENT
    assert call(q=_rows(), q_out=8) == E.WISE_ERR_ALIGNMENT
    assert call(flags=2) == E.WISE_ERR_INVALID_ARGUMENT
    for r in (-16, 8, 24, 80):
        assert call(rotary=r) == E.WISE_ERR_INVALID_ARGUMENT, r
    assert call(rope=None) == E.WISE_ERR_INVALID_ARGUMENT
    assert call(rope=20) == E.WISE_ERR_ALIGNMENT
    assert call(k=_rows(None)) == E.WISE_ERR_INVALID_ARGUMENT
    assert call(k=_rows(8)) == E.WISE_ERR_ALIGNMENT
    assert call(v=_rows(strides=(64, 4, 64))) == E.WISE_ERR_ALIGNMENT
    assert call(v=_rows(strides=(64, -64, 64))) == E.WISE_ERR_INVALID_ARGUMENT
    assert call(new_len=2) == E.WISE_ERR_ALIGNMENT
    assert call(positions=3) == E.WISE_ERR_ALIGNMENT
    assert call(n=1 << 30) == E.WISE_ERR_UNSUPPORTED                   # batch * n past 32 bits
    assert lib.wise_cache_append(_cache(), 3, None, _rows(), 0, None, None, None, None, None, 0, 0, None) == \
        E.WISE_ERR_INVALID_ARGUMENT


def test_tree_attention_arguments(lib):
    ws = lib.wise_attn_tree_workspace(_cache(), 4, 3)
    assert ws > 0

    def call(c=None, heads=4, n=3, q=None, new_len=None, mask=None, scale=0.0, dtype=0, o=16, lse=None, w=16, wb=ws):
        return lib.wise_attn_tree(c or _cache(), heads, n, q or _rows(), new_len, mask, scale, dtype, o, lse, w, wb, None)
    assert call(heads=3) == E.WISE_ERR_INVALID_ARGUMENT
    assert call(heads=0) == E.WISE_ERR_INVALID_ARGUMENT
    assert call(n=0) == E.WISE_ERR_INVALID_ARGUMENT
    assert call(n=129) == E.WISE_ERR_UNSUPPORTED
    assert call(dtype=2) == E.WISE_ERR_INVALID_ARGUMENT
    assert call(scale=-1.0) == E.WISE_ERR_INVALID_ARGUMENT
    assert call(scale=float("inf")) == E.WISE_ERR_INVALID_ARGUMENT
    assert call(scale=float("nan")) == E.WISE_ERR_INVALID_ARGUMENT
    assert call(o=None) == E.WISE_ERR_INVALID_ARGUMENT
    assert call(o=8) == E.WISE_ERR_ALIGNMENT
    assert call(lse=2) == E.WISE_ERR_ALIGNMENT
    assert call(mask=2) == E.WISE_ERR_ALIGNMENT
    assert call(q=_rows(strides=(64, 64, 12))) == E.WISE_ERR_ALIGNMENT
    assert call(w=None) == E.WISE_ERR_WORKSPACE
    assert call(wb=ws - 1) == E.WISE_ERR_WORKSPACE
    assert call(w=8) == E.WISE_ERR_ALIGNMENT
    for bad in (dict(c=_cache(head_dim=32)), dict(heads=5), dict(n=0), dict(n=129)):
        assert lib.wise_attn_tree_workspace(bad.get("c", _cache()), bad.get("heads", 4), bad.get("n", 3)) == 0
    # the workspace query reads no device memory
    assert lib.wise_attn_tree_workspace(_cache(kp=None, vp=None, table=None, lengths=None), 4, 3) == ws
    assert lib.wise_attn_tree_workspace(None, 4, 3) == 0


def test_accept_arguments(lib):
    def call(c=None, tokens=4, path=16, na=16, out=64):
        return lib.wise_cache_accept(c or _cache(), tokens, path, na, out, None)
    assert call(na=None) == E.WISE_ERR_INVALID_ARGUMENT
    assert call(out=None) == E.WISE_ERR_INVALID_ARGUMENT
    assert call(tokens=0) == E.WISE_ERR_INVALID_ARGUMENT
    assert call(path=2) == E.WISE_ERR_ALIGNMENT
    assert call(na=2) == E.WISE_ERR_ALIGNMENT
    assert call(out=66) == E.WISE_ERR_ALIGNMENT
    # the new lengths must not lie over the old ones (2 sequences: 8 bytes)
    for at in (1 << 20, (1 << 20) + 4, (1 << 20) - 4):
        assert call(out=at) == E.WISE_ERR_INVALID_ARGUMENT


def test_accept_refuses_results_over_its_inputs(lib):
    # 2 sequences; a path of 4 tokens: 32 bytes
    def call(out, na=1 << 16, path=1 << 17):
        return lib.wise_cache_accept(_cache(), 4, path, na, out, None)
    for out in (1 << 16, (1 << 16) + 4, (1 << 16) - 4, 1 << 17, (1 << 17) + 28, (1 << 17) - 4):
        assert call(out) == E.WISE_ERR_INVALID_ARGUMENT
    table = _cache().page_table
    assert call(table) == E.WISE_ERR_INVALID_ARGUMENT and call(table + 4) == E.WISE_ERR_INVALID_ARGUMENT


def test_append_refuses_rotated_queries_over_its_inputs(lib):
    # 2 sequences, 3 tokens, 2 heads of 64 (128 bytes a row); queries, keys and
    # values of a token side by side: 6 rows a token, 18 a sequence
    at = 1 << 24

    def call(out, heads=2, q=at, strides=(18 * 64, 64, 6 * 64), **more):
        c = _cache(kp=1 << 20, vp=1 << 21, table=1 << 22, lengths=1 << 23)
        r = [_rows(q + x * 128, strides) for x in (0, 2, 4)]
        args = dict(dict(new_len=1 << 25, positions=1 << 26, rope=1 << 27), **more)
        return lib.wise_cache_append(c, 3, r[1], r[2], heads, r[0], out, args["new_len"], args["positions"], args["rope"], 64,
                                     0, None)
    size = 2 * 2 * 3 * 128
    pool = 8 * 2 * 16 * 64 * 2
    for base, length in ((at, 36 * 128), (1 << 20, pool), (1 << 21, pool), (1 << 22, 32), (1 << 23, 16), (1 << 25, 16),
                         (1 << 26, 32), (1 << 27, 256)):
        for out in (base, base + length - 16, base - size + 16):
            assert call(out) == E.WISE_ERR_INVALID_ARGUMENT, hex(out)
    # every row of the three is found, and nothing between them: the second
    # sequence's rows lie far behind, and each token's are 64 rows apart
    for token in range(3):
        for row in range(6):
            for seq in range(2):
                where = at + seq * (1 << 20) + token * 64 * 128 + row * 128
                assert call(where + 112, strides=(1 << 19, 64, 64 * 64)) == E.WISE_ERR_INVALID_ARGUMENT
                assert call(where - size + 16, strides=(1 << 19, 64, 64 * 64)) == E.WISE_ERR_INVALID_ARGUMENT


def test_tree_attention_refuses_results_over_its_buffers(lib):
    # 2 sequences, 2 heads over 2, 3 tokens of 64 values (128 bytes a row): 1536 bytes of O, 48 of LSE
    kp, vp, table, lengths, q, new_len, mask, o, lse, w = ((1 << 20) * x for x in range(1, 11))
    ws = lib.wise_attn_tree_workspace(_cache(), 2, 3)
    assert 16 < ws < 1 << 20

    def call(**other):
        a = dict(dict(o=o, lse=lse, w=w, dtype=0), **other)
        return lib.wise_attn_tree(_cache(kp=kp, vp=vp, table=table, lengths=lengths), 2, 3, _rows(q, (6 * 64, 64, 128)),
                                  new_len, mask, 0.0, a["dtype"], a["o"], a["lse"], a["w"], ws, None)
    pool = 8 * 2 * 16 * 64 * 2
    for base, length in ((kp, pool), (vp, pool), (table, 32), (lengths, 16), (q, 12 * 128), (new_len, 16), (mask, 32)):
        for name, size, step in (("o", 12 * 128, 16), ("lse", 48, 4), ("w", ws, 16)):
            for at in (base, base + length - 16, base - size + step):
                assert call(**{name: at}) == E.WISE_ERR_INVALID_ARGUMENT, (name, hex(at))
    for at in (o, o + 12 * 128 - 4, o - 44):
        assert call(lse=at) == E.WISE_ERR_INVALID_ARGUMENT
    assert call(dtype=1, lse=o + 24 * 128 - 4) == E.WISE_ERR_INVALID_ARGUMENT  # O of 32 bits: twice as long
    for at in (w, w + ws - 16, w - 12 * 128 + 16):
        assert call(o=at) == E.WISE_ERR_INVALID_ARGUMENT
    for at in (w, w + ws - 4, w - 44):
        assert call(lse=at) == E.WISE_ERR_INVALID_ARGUMENT


def test_pools_that_share_memory_are_refused_where_they_are_written(lib):
    pool = 8 * 2 * 16 * 64 * 2
    for vp in (1 << 20, (1 << 20) + pool - 16, (1 << 20) - pool + 16):
        c = _cache(kp=1 << 20, vp=vp, table=1 << 22, lengths=1 << 23)
        assert lib.wise_cache_append(c, 3, _rows(1 << 24), _rows(1 << 25), 0, None, None, None, None, None, 0, 0, None) == \
            E.WISE_ERR_INVALID_ARGUMENT
        assert lib.wise_cache_accept(c, 4, 1 << 24, 1 << 25, 1 << 26, None) == E.WISE_ERR_INVALID_ARGUMENT


def test_accept_refuses_new_lengths_in_the_pools(lib):
    pool = 8 * 2 * 16 * 64 * 2
    c = _cache(kp=1 << 20, vp=1 << 21, table=1 << 22, lengths=1 << 23)
    for base in (1 << 20, 1 << 21):
        for out in (base, base + pool - 4, base - 4):
            assert lib.wise_cache_accept(c, 4, 1 << 24, 1 << 25, out, None) == E.WISE_ERR_INVALID_ARGUMENT


def test_status_text(lib):
    assert "cache" in lib.wise_status_str(E.WISE_ERR_BAD_CACHE).decode()


def test_structs_match_the_header():
    assert ctypes.sizeof(_lib.PagedCacheDesc) == 64 and ctypes.sizeof(_lib.Rows) == 32


def test_rope_frequencies():
    r = wise.rope_frequencies(64, device="cpu")
    assert r.steps.dtype == torch.int64 and r.steps.numel() == 32 and not r.pairs
    # one radian per position: 1 / (2 pi) turns of 2^64
    assert abs(int(r.steps[0]) / 2.0 ** 64 - 0.15915494309189535) < 1e-16
    assert int(wise.rope_frequencies(16, inv_freq=[-1.0] + [0.0] * 7, device="cpu").steps[0]) == -int(r.steps[0])
    assert wise.rope_frequencies(0, device="cpu").steps.numel() == 0
    for bad in (8, -16, 40):
        with pytest.raises(ValueError):
            wise.rope_frequencies(bad, device="cpu")
    for freq in ([1.0], [float("nan")] * 8, [float("inf")] * 8):
        with pytest.raises(ValueError):
            wise.rope_frequencies(16, inv_freq=freq, device="cpu")


@pytest.mark.parametrize("n", [1, 31, 32, 33, 64, 128])
def test_pack_tree_mask(n):
    g = torch.Generator().manual_seed(n)
    m = torch.rand((2, n, n), generator=g) < 0.5
    p = wise.pack_tree_mask(m)
    assert p.dtype == torch.int32 and p.shape == (2, n, (n + 31) // 32)
    j = torch.arange(n)
    assert torch.equal((p[:, :, j // 32] >> (j % 32).int()) & 1 == 1, m)
    if n % 32:
        assert torch.all((p[:, :, -1].long() & 0xffffffff) >> (n % 32) == 0)
    with pytest.raises(ValueError):
        wise.pack_tree_mask(m.int())
    with pytest.raises(ValueError):
        wise.pack_tree_mask(m[0])


def _cpu_cache():
    pool = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    return wise.PagedCache(pool, pool.clone(), torch.zeros((2, 2), dtype=torch.int32), torch.zeros(2, dtype=torch.int32))


def test_host_tensors_are_refused():
    c = _cpu_cache()
    rows = torch.zeros((2, 2, 3, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        wise.cache_append(c, rows, rows)
    with pytest.raises(ValueError, match="CUDA"):
        wise.tree_attention(rows, c)
    with pytest.raises(ValueError, match="CUDA"):
        wise.cache_accept(c, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="PagedCache"):
        wise.cache_accept(None, torch.zeros(2, dtype=torch.int32))


def test_row_checks():
    dev = -1  # the checks below fail or pass before any device is asked
    ok = torch.zeros((2, 2, 3, 64), dtype=torch.bfloat16)
    for bad in (ok.float(), ok[0]):
        with pytest.raises(ValueError, match="bfloat16"):
            wise._check_rows("k", bad, 2, 2, 64, dev)
    with pytest.raises(ValueError, match="device"):
        wise._check_rows("k", ok, 2, 2, 64, dev)
    with pytest.raises(ValueError, match="shape"):
        wise._check_array("new_len", torch.zeros(3, dtype=torch.int32), torch.int32, (2,), dev)
    with pytest.raises(ValueError, match="shape"):
        wise._check_array("new_len", torch.zeros(2, dtype=torch.int64), torch.int32, (2,), dev)
    with pytest.raises(ValueError, match="device"):
        wise._check_array("new_len", torch.zeros(2, dtype=torch.int32), torch.int32, (2,), dev)


def test_axes_past_32_bits_are_refused():
    """Not cut off to their low bits: 2^32 + 1 tokens are not one."""
    long = (1 << 32) + 1
    row = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16)
    for shape in ((1, 1, long, 64), (1, long, 1, 64)):
        with pytest.raises(ValueError, match="2\\^31"):
            wise._check_rows("k", row.expand(shape), 1, None, 64, -1)
    pool = torch.zeros((1, 1, 16, 64), dtype=torch.bfloat16)
    for table in ((1, long), (long, 1)):
        c = wise.PagedCache(pool, pool.clone(), torch.empty(table, dtype=torch.int32, device="meta"), torch.zeros(1, dtype=torch.int32))
        with pytest.raises(ValueError, match="2\\^31"):
            wise._check_cache(c)
