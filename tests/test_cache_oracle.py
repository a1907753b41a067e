"""Pins of the paged-cache oracle (no GPU): closed forms, torch's fp64
attention with an explicit mask, and the whole loop of append, attention and
acceptance against plain causal attention of the kept tokens."""
import math

import numpy as np
import pytest
import torch

from oracle import cache_oracle as C


def test_rotation_is_a_complex_product():
    rng = np.random.default_rng(0)
    x = rng.standard_normal(24)
    f = np.array([1.0, 0.3, 0.01, 1e-4])
    pos = 12345
    w = np.exp(1j * pos * f)
    z = (x[:4] + 1j * x[4:8]) * w
    y = C.rotate(x, pos, f, pairs=False)
    assert np.allclose(y[:8], np.concatenate([z.real, z.imag]), atol=1e-11) and np.array_equal(y[8:], x[8:])
    z = (x[0:8:2] + 1j * x[1:8:2]) * w
    y = C.rotate(x, pos, f, pairs=True)
    assert np.allclose(y[0:8:2], z.real, atol=1e-11) and np.allclose(y[1:8:2], z.imag, atol=1e-11)
    assert np.array_equal(C.rotate(x, 0, f, False), x)


def test_rotated_scores_depend_on_the_distance_alone():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 16))
    f = 10000.0 ** (-np.arange(8) / 8)
    s = [C.rotate(q, a, f, True) @ C.rotate(k, b, f, True) for a, b in ((7, 2), (1007, 1002), (5, 0))]
    assert np.allclose(s, s[0], atol=1e-9)


@pytest.mark.parametrize("page", [16, 32])
def test_attention_equals_torch_with_a_mask(page):
    rng = np.random.default_rng(page)
    b, h, hk, n, d = 2, 4, 2, 5, 64
    lengths, news = [37, 0], [5, 3]
    table = np.array([[3, 1, 0], [2, 4, 5]], np.int32)
    kp, vp = rng.standard_normal((2, 6, hk, page, d))
    q = rng.standard_normal((b, h, n, d))
    sees = rng.random((b, n, n)) < 0.5
    sees[1, 1] = False  # behind nothing: an empty row
    o, lse, _, _ = C.tree_attention(q, kp, vp, table, lengths, sees, news)
    for s in range(b):
        total = lengths[s] + news[s]
        at = np.array([[table[s][t // page], t % page] for t in range(total)])
        k, v = (torch.from_numpy(x[at[:, 0], :, at[:, 1]].transpose(1, 0, 2)) for x in (kp, vp))
        mask = np.concatenate([np.ones((news[s], lengths[s]), bool), sees[s, :news[s], :news[s]]], 1)
        want = torch.nn.functional.scaled_dot_product_attention(
            torch.from_numpy(q[s, :, :news[s]]), k.repeat_interleave(h // hk, 0), v.repeat_interleave(h // hk, 0),
            attn_mask=torch.from_numpy(mask)).numpy()
        full = mask.any(1)
        assert np.allclose(o[s, :, :news[s]][:, full], want[:, full], atol=1e-12)
        assert np.all(o[s, :, :news[s]][:, ~full] == 0) and np.all(lse[s, :, :news[s]][:, ~full] == -np.inf)
    assert np.all(o[1, :, 3:] == 0) and np.all(lse[1, :, 3:] == -np.inf)


def test_lse_of_zero_queries_counts_tokens():
    page, d = 16, 64
    kp = np.ones((2, 1, page, d))
    vp = np.tile(np.arange(page, dtype=float)[None, None, :, None], (2, 1, 1, d))
    o, lse, _, _ = C.tree_attention(np.zeros((1, 1, 2, d)), kp, vp, [[1, 0]], [3], np.tril(np.ones((1, 2, 2), bool)))
    assert np.allclose(lse[0, 0], [math.log(4), math.log(5)]) and np.allclose(o[0, 0, :, 0], [1.5, 2.0])


def test_append_attend_accept_equals_plain_causal_attention():
    """A drafted tree is appended with its depths as positions, one path is
    accepted, and the next token sees what a plain sequence would hold."""
    rng = np.random.default_rng(3)
    page, d, f = 16, 64, 10000.0 ** (-np.arange(32) / 32)
    table, kp, vp = [[2, 0, 1]], np.zeros((3, 1, page, d)), np.zeros((3, 1, page, d))
    k, v = rng.standard_normal((2, 1, 1, 14, d))
    kp, vp = C.append(kp, vp, table, [0], k, v, inv_freq=f)
    # tokens 0-1-3 are the path kept; 2 and 4 are other branches
    parent = [-1, 0, 0, 1, 2]
    depth, sees = [], np.zeros((1, 5, 5), bool)
    for i, p in enumerate(parent):
        depth.append(0 if p < 0 else depth[p] + 1)
        if p >= 0:
            sees[0, i] = sees[0, p]
        sees[0, i, i] = True
    dk, dv = rng.standard_normal((2, 1, 1, 5, d))
    kp, vp = C.append(kp, vp, table, [14], dk, dv, positions=[[14 + x for x in depth]], inv_freq=f)
    q = rng.standard_normal((1, 1, 5, d))
    o, _, _, _ = C.tree_attention(q, kp, vp, table, [14], sees)
    kp, vp, lengths = C.accept(kp, vp, table, [14], [3], [[0, 1, 3]])
    assert list(lengths) == [17]
    seq_k = np.concatenate([k[0, 0], dk[0, 0, [0, 1, 3]]])
    seq_v = np.concatenate([v[0, 0], dv[0, 0, [0, 1, 3]]])
    rot = np.array([C.rotate(x, t, f, False) for t, x in enumerate(seq_k)])
    for t in range(17):
        pg, row = C.slot(table, 0, t, page)
        assert np.allclose(kp[pg, 0, row], rot[t], atol=1e-12) and np.array_equal(vp[pg, 0, row], seq_v[t])
    for at, i in ((14, 0), (15, 1), (16, 3)):
        s = rot[:at + 1] @ q[0, 0, i] / math.sqrt(d)
        p = np.exp(s - s.max())
        assert np.allclose(o[0, 0, i], p @ seq_v[:at + 1] / p.sum(), atol=1e-12)
