"""Plain fp64 restatement of the paged-cache operators (test infrastructure
only, sharing no code with the CUDA path): the append with its position
rotation, attention of drafted tokens over the cache, and the acceptance of a
drafted path. NumPy, one sequence at a time."""
from __future__ import annotations

import math

import numpy as np


def slot(page_table, b, t, page):
    """(page, row) of token t of sequence b."""
    return int(page_table[b][t // page]), t % page


def rotate(x, position, inv_freq, pairs):
    """One head's values x [d] rotated by its position (fp64): the first
    2 len(inv_freq) values, in neighbouring pairs or as two halves."""
    y = np.array(x, np.float64)
    half = len(inv_freq)
    for i, f in enumerate(inv_freq):
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
        # reduced before the sine: positions times frequencies are far from 0
        angle = math.fmod(float(position) * float(f), 2.0 * math.pi)
        c, s = math.cos(angle), math.sin(angle)
        y[a], y[b] = x[a] * c - x[b] * s, x[b] * c + x[a] * s
    return y


def append(k_pages, v_pages, page_table, lengths, k, v, new_len=None, positions=None, inv_freq=(), pairs=False):
    """The pools after the append, as fp64 copies."""
    kp, vp = np.array(k_pages, np.float64), np.array(v_pages, np.float64)
    page = kp.shape[2]
    b, hk, n, _ = k.shape
    for s in range(b):
        for i in range(n if new_len is None else int(new_len[s])):
            pg, row = slot(page_table, s, int(lengths[s]) + i, page)
            pos = int(lengths[s]) + i if positions is None else int(positions[s][i])
            for h in range(hk):
                kp[pg, h, row] = rotate(k[s, h, i], pos, inv_freq, pairs)
                vp[pg, h, row] = v[s, h, i]
    return kp, vp


def tree_attention(q, k_pages, v_pages, page_table, lengths, sees, new_len=None, scale=None):
    """(O, LSE, sum of the weights times |v|, largest sum of |q k| of a row's
    scores) of q [batch, heads, n, d]; sees [batch, n, n] boolean: token i sees
    drafted token j."""
    b, h, n, d = q.shape
    hk, page = k_pages.shape[1], k_pages.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out = np.zeros(q.shape)
    weight = np.zeros(q.shape)
    lse = np.full((b, h, n), -np.inf)
    size = np.zeros((b, h, n))
    for s in range(b):
        length, m = int(lengths[s]), n if new_len is None else int(new_len[s])
        at = [slot(page_table, s, t, page) for t in range(length + m)]
        for x in range(hk):
            kk = np.array([k_pages[pg, x, row] for pg, row in at], np.float64).reshape(-1, d)
            vv = np.array([v_pages[pg, x, row] for pg, row in at], np.float64).reshape(-1, d)
            for y in range(x * (h // hk), (x + 1) * (h // hk)):
                for i in range(m):
                    seen = np.concatenate([np.arange(length), length + np.nonzero(sees[s, i, :m])[0]]).astype(int)
                    if len(seen) == 0:
                        continue
                    qi = np.asarray(q[s, y, i], np.float64)
                    sc = kk[seen] @ qi * scale
                    top = sc.max()
                    p = np.exp(sc - top)
                    out[s, y, i] = p @ vv[seen] / p.sum()
                    weight[s, y, i] = p @ np.abs(vv[seen]) / p.sum()
                    lse[s, y, i] = top + math.log(p.sum())
                    size[s, y, i] = (np.abs(kk[seen]) @ np.abs(qi)).max() * scale
    return out, lse, weight, size


def accept(k_pages, v_pages, page_table, lengths, n_accepted, path):
    """The pools after the move and the new lengths."""
    kp, vp = np.array(k_pages, np.float64), np.array(v_pages, np.float64)
    page = kp.shape[2]
    for s in range(len(lengths)):
        for i in range(int(n_accepted[s])):
            if path is None:
                continue
            a, b = slot(page_table, s, int(lengths[s]) + int(path[s][i]), page), slot(page_table, s, int(lengths[s]) + i, page)
            kp[b[0], :, b[1]] = kp[a[0], :, a[1]].copy()
            vp[b[0], :, b[1]] = vp[a[0], :, a[1]].copy()
    return kp, vp, np.asarray(lengths) + np.asarray(n_accepted)
