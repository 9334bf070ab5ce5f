"""Per-head norms with the rotation, their gradient, and paged key/value caches (fp64 oracle).
TEST INFRASTRUCTURE ONLY: tests use it; the CUDA library never does.

The rotation is that of msa_docs.py.  The norm is the root-mean-square norm of one head's d
elements with a weight per element; a paged cache holds token p of sequence s in row
p % page of page table[s][p // page]."""
from __future__ import annotations

import numpy as np

from .msa_docs import rope_angles

__all__ = ["rotate_heads", "norm_rope", "norm_rope_backward", "paged_positions",
           "paged_append", "paged_attention"]


def rotate_heads(x, pos, base, inverse=False):
    """x [T, h, d] rotated to positions pos [T] (by the negated angles when inverse)."""
    half = x.shape[-1] // 2
    ang = rope_angles(np.asarray(pos), x.shape[-1], base)
    c, s = np.cos(ang)[:, None, :], np.sin(ang)[:, None, :]
    if inverse:
        s = -s
    a, b = x[..., :half].astype(np.float64), x[..., half:].astype(np.float64)
    return np.concatenate([a * c - b * s, b * c + a * s], axis=-1)


def norm_heads(x, w, eps):
    """RMS norm of the last axis, times w."""
    x = x.astype(np.float64)
    r = 1.0 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    return x * r * (1.0 if w is None else np.asarray(w, np.float64))


def norm_rope(x, w, pos, base, eps):
    return rotate_heads(norm_heads(x, w, eps), pos, base)


def norm_rope_backward(dy, x, w, pos, base, eps):
    """(dx, dw) of norm_rope for the upstream gradient dy."""
    x = x.astype(np.float64)
    r = 1.0 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    g = rotate_heads(dy, pos, base, inverse=True)
    u = g if w is None else g * np.asarray(w, np.float64)
    dx = r * (u - r ** 2 * x * (u * x).mean(-1, keepdims=True))
    return dx, (g * r * x).sum((0, 1))


def paged_positions(kv_lens, cu):
    """[(packed token, sequence, position)] of a step's new tokens."""
    out = []
    for s, L in enumerate(kv_lens):
        n = cu[s + 1] - cu[s]
        out += [(cu[s] + i, s, L - n + i) for i in range(n)]
    return out


def paged_append(k_pages, v_pages, k, v, table, kv_lens, cu, page, base=None, wk=None, eps=None):
    """The pools (float64 copies) after the step's tokens went in; tokens without a page are
    left out."""
    kp, vp = k_pages.astype(np.float64), v_pages.astype(np.float64)
    for t, s, pos in paged_positions(kv_lens, cu):
        if pos < 0 or pos >= table.shape[1] * page:
            continue
        pg = table[s, pos // page]
        if not 0 <= pg < kp.shape[0]:
            continue
        row = k[t:t + 1].astype(np.float64)
        if eps is not None:
            row = norm_heads(row, wk, eps)
        if base is not None:
            row = rotate_heads(row, [pos], base)
        kp[pg, :, pos % page] = row[0]
        vp[pg, :, pos % page] = v[t]
    return kp, vp


def paged_attention(q, k_pages, v_pages, table, kv_lens, cu, page, scale):
    """(o [T, hq, d], lse [T, hq], a [T, hq, d], s [T, hq]) of the step's tokens: causal
    attention over each sequence's cache.  a = sum_i softmax_i |v_i| and s = the largest
    |scale| * sum |q_j k_ij| of a visible key are what error bounds are made of.  Rows of no
    sequence stay NaN; a row that sees nothing has o = 0, lse = -inf.  A table entry that is
    no page reads as zeros; keys past the table row do not exist."""
    T, hq, d = q.shape
    hkv = k_pages.shape[1]
    G = hq // hkv
    o, a = np.full((T, hq, d), np.nan), np.full((T, hq, d), np.nan)
    lse, big = np.full((T, hq), np.nan), np.zeros((T, hq))
    q = q.astype(np.float64)
    for s, L in enumerate(kv_lens):
        n = cu[s + 1] - cu[s]
        have = max(0, min(L, table.shape[1] * page))
        K, V = np.zeros((have, hkv, d)), np.zeros((have, hkv, d))
        for p0 in range(0, have, page):
            pg, m = table[s, p0 // page], min(page, have - p0)
            if 0 <= pg < k_pages.shape[0]:
                K[p0:p0 + m] = k_pages[pg, :, :m].transpose(1, 0, 2)
                V[p0:p0 + m] = v_pages[pg, :, :m].transpose(1, 0, 2)
        for i in range(n):
            t, see = cu[s] + i, max(0, min(L - n + i + 1, have))
            if see == 0:
                o[t], a[t], lse[t] = 0.0, 0.0, -np.inf
                continue
            for h in range(hq):
                x = scale * (K[:see, h // G] @ q[t, h])
                m = x.max()
                p = np.exp(x - m)
                l = p.sum()
                o[t, h] = p @ V[:see, h // G] / l
                a[t, h] = p @ np.abs(V[:see, h // G]) / l
                lse[t, h] = m + np.log(l)
                big[t, h] = abs(scale) * (np.abs(K[:see, h // G]) @ np.abs(q[t, h])).max()
    return o, lse, a, big
