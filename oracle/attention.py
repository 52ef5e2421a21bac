"""float64 definitions of the attention operators (include/gdn_attention.h): numpy, one token after another.

TEST INFRASTRUCTURE ONLY, like the rest of this package: no code is shared with the CUDA library.  Pools are
[n_pages, page_size, Hkv, d]; slot s of request b is row s % page_size of page table[b][s // page_size].
"""
from __future__ import annotations

import numpy as np


def _f64(x):
    return np.asarray(x, dtype=np.float64)


def slot(table, b, s, page_size):
    return int(table[b][s // page_size]), s % page_size


def turn(x, cos_sin, position, interleaved=False):
    """Row(s) x [..., d] turned by the angles of a position."""
    rot = cos_sin.shape[1]
    half = rot // 2
    y = _f64(x).copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = float(cos_sin[position, i]), float(cos_sin[position, half + i])
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def normed(x, weight, eps):
    x = _f64(x)
    return x if weight is None else x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * _f64(weight)


def append(q, k, v, k_cache, v_cache, table, lens, offsets=None, depth=None, cos_sin=None, interleaved=False, q_weight=None,
           k_weight=None, eps=1e-6):
    """(q_out, k_cache, v_cache); rows of q_out that are left out are NaN."""
    q, k, v, kc, vc = _f64(q), _f64(k), _f64(v), _f64(k_cache).copy(), _f64(v_cache).copy()
    B, page = len(lens), kc.shape[1]
    offsets = range(B + 1) if offsets is None else offsets
    out = np.full(q.shape, np.nan)
    for b in range(B):
        if lens[b] < 0:
            continue
        for t in range(int(offsets[b]), int(offsets[b + 1])):
            i = t - int(offsets[b])
            position = int(lens[b]) + (i if depth is None else int(depth[t]) - 1)
            x, y = normed(q[t], q_weight, eps), normed(k[t], k_weight, eps)
            if cos_sin is not None:
                x, y = turn(x, cos_sin, position, interleaved), turn(y, cos_sin, position, interleaved)
            p, r = slot(table, b, int(lens[b]) + i, page)
            out[t], kc[p, r], vc[p, r] = x, y, v[t]
    return out, kc, vc


def softmax_rows(q, k, v, seen, scale):
    """One head: q [n, d] over k, v [m, d], seen [n, m]; zeros where nothing is seen."""
    o = np.zeros(q.shape)
    for i in range(q.shape[0]):
        at = np.nonzero(seen[i])[0]
        if not len(at):
            continue
        with np.errstate(invalid="ignore"):
            x = scale * (k[at] @ q[i])
            e = np.exp(x - np.max(x))
            o[i] = (e / e.sum()) @ v[at]
    return o


def bits(mask, n):
    """[T, n] booleans of the first n bits of each row of int32 or uint32 words."""
    words = np.asarray(mask).astype(np.int64) & 0xFFFFFFFF
    j = np.arange(n)
    return ((words[:, j // 32] >> (j % 32)) & 1).astype(bool)


def attend(q, k_cache, v_cache, table, lens, offsets=None, mask=None, scale=1.0):
    """o [T, Hq, d]; offsets None: one token a request."""
    q, kc, vc = _f64(q), _f64(k_cache), _f64(v_cache)
    B, page, hkv, group = len(lens), kc.shape[1], kc.shape[2], q.shape[1] // kc.shape[2]
    offsets = range(B + 1) if offsets is None else offsets
    o = np.zeros(q.shape)
    for b in range(B):
        lo, hi = int(offsets[b]), int(offsets[b + 1])
        n, ln = hi - lo, int(lens[b])
        if ln < 0 or n == 0:
            continue
        at = [slot(table, b, s, page) for s in range(ln + n)]
        pages, rows = [a[0] for a in at], [a[1] for a in at]
        seen = np.ones((n, ln + n), dtype=bool)
        seen[:, ln:] = np.tril(np.ones((n, n), dtype=bool)) if mask is None else bits(mask[lo:hi], n)
        for h in range(hq := q.shape[1]):
            assert hq % hkv == 0
            o[lo:hi, h] = softmax_rows(q[lo:hi, h], kc[pages, rows, h // group], vc[pages, rows, h // group], seen, scale)
    return o


def commit(k_cache, v_cache, table, lens, path_offsets, path):
    kc, vc = np.array(k_cache), np.array(v_cache)
    page, new = kc.shape[1], np.array(lens).copy()
    for b in range(len(lens)):
        if lens[b] < 0:
            continue
        mine = path[path_offsets[b]:path_offsets[b + 1]]
        src = [slot(table, b, int(lens[b]) + int(j), page) for j in mine]
        rows = [(kc[s].copy(), vc[s].copy()) for s in src]
        for i, (x, y) in enumerate(rows):
            to = slot(table, b, int(lens[b]) + i, page)
            kc[to], vc[to] = x, y
        new[b] = lens[b] + len(mine)
    return kc, vc, new
