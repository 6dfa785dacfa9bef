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
