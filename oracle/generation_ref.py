"""Float64 numpy statement of the calls around the key-value cache (test
infrastructure only): per-head RMSNorm with rotary positions and its gradient,
the page plan, attention of one new token.  Explicit and slow; shares no code
with the CUDA library."""
from __future__ import annotations

import math

import numpy as np

from .adaspark_ref import _f64


def rope_pairs(d, rot, interleaved):
    """Elements (first, second) of the rotated pairs."""
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rope_angles(positions, freq, sections=None):
    """Angles [N, rot/2]: positions [N], or [3, N] with the pairs per axis."""
    pos = np.asarray(positions, dtype=np.float64)
    freq = np.asarray(freq, dtype=np.float64)
    if sections is None:
        return pos[:, None] * freq
    axis = np.repeat(np.arange(3), sections)
    return pos[axis].T * freq


def rotate(x, angles, rot, interleaved, magnitude=1.0):
    """The rotation of [N, h, d] heads; a negative angle and the same magnitude
    give its transpose."""
    y = _f64(x).copy()
    f, s = rope_pairs(y.shape[-1], rot, interleaved)
    c, sn = magnitude * np.cos(angles)[:, None], magnitude * np.sin(angles)[:, None]
    a, b = y[..., f].copy(), y[..., s].copy()
    y[..., f] = a * c - b * sn
    y[..., s] = b * c + a * sn
    return y


def head_norm(x, w, eps):
    """(x / sqrt(mean(x^2) + eps) * w, the inverse roots); x itself without w."""
    x = _f64(x)
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    return (x, r) if w is None else (x * r * _f64(w), r)


def qk_rope(x, angles, rot, interleaved, w=None, eps=1e-6, magnitude=1.0):
    """One of queries and keys: norm, then rotation."""
    return rotate(head_norm(x, w, eps)[0], angles, rot, interleaved, magnitude)


def qk_rope_backward(dy, x, angles, rot, interleaved, w=None, eps=1e-6, magnitude=1.0):
    """(dx, dw) of qk_rope; dw is None without w."""
    g = rotate(dy, -angles, rot, interleaved, magnitude)
    if w is None:
        return g, None
    _, r = head_norm(x, w, eps)
    xhat = _f64(x) * r
    gw = g * _f64(w)
    dx = r * (gw - xhat * np.mean(gw * xhat, axis=-1, keepdims=True))
    return dx, (g * xhat).sum(axis=(0, 1))


def kv_plan(old, new, table, free, n_free, page_size, n_rows):
    """One step on copies: returns (table, free, n_free, slots, positions, starts),
    or None for a plan that cannot be carried out.  A list of pages stands for the
    free list: gifts are appended in reverse order, takes pop its end."""
    table, free = np.array(table), np.array(free)
    pages = lambda n: -(-int(n) // page_size)  # noqa: E731
    if any(n < 0 or pages(n) > table.shape[1] for n in list(old) + list(new)):
        return None
    if not 0 <= n_free <= len(free):
        return None
    stack = [int(p) for p in free[:n_free]]
    gifts = []
    for i, (o, n) in enumerate(zip(old, new)):
        gifts += [int(p) for p in table[i, pages(n):pages(o)]]
    stack += gifts[::-1]
    slots, positions, starts = [], [], [0]
    for i, (o, n) in enumerate(zip(old, new)):
        for j in range(pages(o), pages(n)):
            if not stack:
                return None
            table[i, j] = stack.pop()
        for t in range(int(o), int(n)):
            slots.append(int(table[i, t // page_size]) * page_size + t % page_size)
            positions.append(t)
        starts.append(len(slots))
    if len(slots) > n_rows or len(stack) > len(free):
        return None
    # entries of the list that stay free beyond the old ones are written, others kept
    free[:len(stack)] = stack
    pad = n_rows - len(slots)
    return table, free, len(stack), slots + [-1] * pad, positions + [0] * pad, starts


def decode_attn(q, k_cache, v_cache, table, lens, scale=None):
    """out [n, hq, d] and lse [n, hq] of one new token per sequence over the
    cache [pages, page_size, hkv, d]; absent pages (outside the cache) hold no keys."""
    q = _f64(q)
    n, hq, d = q.shape
    n_pages, page_size, hkv = (int(x) for x in k_cache.shape[:3])
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out, lse = np.zeros((n, hq, d)), np.full((n, hq), -np.inf)
    table = np.asarray(table)
    for i in range(n):
        j = np.arange(int(lens[i]))
        page, off = table[i, j // page_size], j % page_size
        there = (page >= 0) & (page < n_pages)
        page, off = page[there], off[there]
        if page.size == 0:
            continue
        k, v = _f64(k_cache[page, off]), _f64(v_cache[page, off])
        for h in range(hq):
            z = k[:, h // (hq // hkv)] @ q[i, h] * scale
            top = z.max()
            if np.isneginf(top):
                continue
            e = np.exp(z - top)
            lse[i, h] = top + math.log(e.sum())
            out[i, h] = (e / e.sum()) @ v[:, h // (hq // hkv)]
    return out, lse
