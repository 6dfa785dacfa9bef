"""fp64 reference of the operators around attention: per-head RMS norm, rotary positions, their
gradients, the paged cache and attention over it (numpy, one plain loop per sequence)."""

from __future__ import annotations

import numpy as np


def rotate(y, pos, inv_freq, interleaved=False, amplitude=1.0, inverse=False):
    """Rotation of the first 2 len(inv_freq) elements of rows y [tokens, heads, d] at positions
    pos [tokens]; inverse: its transpose."""
    y = np.array(y, dtype=np.float64)
    half = len(inv_freq)
    ang = np.asarray(pos, dtype=np.float64)[:, None, None] * np.asarray(inv_freq, np.float64)
    c, s = amplitude * np.cos(ang), amplitude * np.sin(ang)
    if inverse:
        s = -s
    one = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    two = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    a, b = y[..., one].copy(), y[..., two].copy()
    y[..., one] = a * c - b * s
    y[..., two] = a * s + b * c
    return y


def rms_norm(x, w, eps):
    x = np.asarray(x, dtype=np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)


def norm_rope(x, pos, w=None, eps=1e-6, inv_freq=None, interleaved=False, amplitude=1.0):
    y = np.asarray(x, np.float64) if w is None else rms_norm(x, w, eps)
    return y if inv_freq is None else rotate(y, pos, inv_freq, interleaved, amplitude)


def norm_rope_backward(dz, x, pos, w=None, eps=1e-6, inv_freq=None, interleaved=False,
                       amplitude=1.0):
    """(dx, dw or None, sum of |terms| of dw) of norm_rope."""
    g = np.asarray(dz, np.float64)
    if inv_freq is not None:
        g = rotate(g, pos, inv_freq, interleaved, amplitude, inverse=True)
    if w is None:
        return g, None, None
    x = np.asarray(x, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh, u = x * r, g * np.asarray(w, np.float64)
    terms = g * xh
    dx = r * (u - xh * (u * xh).mean(-1, keepdims=True))
    return dx, terms.sum((0, 1)), np.abs(terms).sum((0, 1))


def paged_keys(cache, table_row, n):
    """[Hkv, n, d] float64: the first n keys of one block-table row of [pages, Hkv, page, d]."""
    page = cache.shape[2]
    out = np.zeros((cache.shape[1], n, cache.shape[3]))
    for i in range(0, n, page):
        m = min(page, n - i)
        out[:, i:i + m] = cache[int(table_row[i // page])][:, :m].astype(np.float64)
    return out


def attend(q, k, v, scale, limits):
    """Attention of q [t, H, d] over k, v [Hkv, n, d]; row i sees keys < limits[i].  Returns
    O [t, H, d], LSE [t, H], the same sum with |v| (for error bounds) and sum |q_e k_e| maxima."""
    t, H, d = q.shape
    G = H // k.shape[0]
    O, A = np.zeros((t, H, d)), np.zeros((t, H, d))
    LSE, size = np.full((t, H), -np.inf), np.zeros((t, H))
    for i in range(t):
        m = int(max(0, min(limits[i], k.shape[1])))
        if m == 0:
            continue
        for h in range(H):
            kk, vv = k[h // G, :m], v[h // G, :m]
            s = scale * (kk @ q[i, h])
            top = s.max()
            p = np.exp(s - top)
            total = p.sum()
            LSE[i, h] = top + np.log(total)
            O[i, h] = (p / total) @ vv
            A[i, h] = (p / total) @ np.abs(vv)
            size[i, h] = scale * (np.abs(kk) @ np.abs(q[i, h])).max()
    return O, LSE, A, size


def attend_where(q, k, v, scale, seen):
    """attend() where row i sees the keys j with seen[i, head of k, j] (seen [t, Hkv or 1, n])."""
    t, H, d = q.shape
    Hkv, n = k.shape[:2]
    O, A = np.zeros((t, H, d)), np.zeros((t, H, d))
    LSE, size = np.full((t, H), -np.inf), np.zeros((t, H))
    seen = np.broadcast_to(seen, (t, Hkv, n))
    for h in range(H):
        kk, vv, there = k[h * Hkv // H], v[h * Hkv // H], seen[:, h * Hkv // H]
        s = np.where(there, scale * (q[:, h] @ kk.T), -np.inf)
        some = there.any(1)
        top = np.where(some, s.max(1, initial=-np.inf), 0.0)
        p = np.exp(s - top[:, None])
        total = p.sum(1)
        with np.errstate(divide="ignore"):
            LSE[:, h] = top + np.log(total)
        p = p / np.where(some, total, 1.0)[:, None]
        O[:, h], A[:, h] = p @ vv, p @ np.abs(vv)
        size[:, h] = scale * np.where(there, np.abs(q[:, h]) @ np.abs(kk).T, 0.0).max(1, initial=0.0)
    return O, LSE, A, size


def tree_sees(parents):
    """[n, n] bool: token i sees itself and its ancestors."""
    n = len(parents)
    out = np.zeros((n, n), dtype=bool)
    for i in range(n):
        j = i
        while j >= 0:
            out[i, j] = True
            j = parents[j]
    return out


def page_bounds(k, page):
    """Smallest and largest of each element of each page's keys: k [Hkv, n, d] -> two [Hkv, pages, d]."""
    cut = [k[:, i:i + page] for i in range(0, k.shape[1], page)]
    return np.stack([c.min(1) for c in cut], 1), np.stack([c.max(1) for c in cut], 1)


def page_scores(q, lo, hi):
    """[Hkv, pages]: the largest of the bounds on q.k over the heads of a group; q [H, d]."""
    Hkv = lo.shape[0]
    x = q.reshape(Hkv, -1, 1, q.shape[1])
    with np.errstate(invalid="ignore"):
        s = (np.maximum(x, 0) * hi[:, None] + np.minimum(x, 0) * lo[:, None]).sum(-1)
    return np.where(np.isnan(s), np.inf, s).max(1)


def largest(values, count):
    """Indices of the `count` largest values, ties to the lowest index, ascending."""
    return np.sort(np.lexsort((np.arange(len(values)), -np.asarray(values)))[:count])


def select_pages(scores, pages, top, first, last):
    """The pages of one query and key/value head: the first and last, and of the others the best."""
    if pages <= top:
        return np.arange(pages)
    mid = first + largest(scores[first:pages - last], top - first - last)
    return np.concatenate([np.arange(first), mid, np.arange(pages - last, pages)])


def key_weights(q, k, scale, lse, limits):
    """[Hkv, n]: the weights exp(scale q.k - lse) of each key summed over queries, and a bound on
    the sum of |terms| times (1 + the size of their exponents); q [t, H, d], lse [t, H]."""
    Hkv, n = k.shape[:2]
    G = q.shape[1] // Hkv
    w, err = np.zeros((Hkv, n)), np.zeros((Hkv, n))
    for i in range(q.shape[0]):
        m = int(max(0, min(limits[i], n)))
        for h in range(q.shape[1]):
            if m == 0 or lse[i, h] == -np.inf:
                continue
            kk = k[h // G, :m]
            p = np.exp(scale * (kk @ q[i, h]) - lse[i, h])
            w[h // G, :m] += p
            err[h // G, :m] += p * (1 + scale * (np.abs(kk) @ np.abs(q[i, h])) + abs(lse[i, h]))
    return w, err


def evict(weights, n, budget, recent):
    """Indices of the keys of one sequence and head that stay, ascending."""
    if n <= budget:
        return np.arange(n)
    w, nan = weights[:n - recent], np.isnan(weights[:n - recent])  # a NaN is above infinity
    best = np.lexsort((np.arange(len(w)), -np.where(nan, np.inf, w), ~nan))[:budget - recent]
    return np.concatenate([np.sort(best), np.arange(n - recent, n)])
