"""Oracle for the attention layers in serving: head norms with rotation, grouped causal attention
over packed prompts, attention of single tokens over a paged cache with a shared prefix.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``). fp64 throughout, from the definitions. Besides
its result each attention function returns sum_j p_j |v_j|, the scale of a rounding of the weights.
"""
from __future__ import annotations

import numpy as np

from .scan import as_f64


def norm_rope(x, w, positions, rot, base=10000.0, eps=1e-6):
    """x [T, H, d] -> (y, bound): y normalised per head, times w (or None), its first rot elements
    turned in pairs (i, i + rot/2) by positions[t] base^(-2i/rot). bound: the sum of the magnitudes
    of the one or two terms of each element."""
    x = as_f64(x)
    xn = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if w is not None:
        xn = xn * as_f64(w)
    y, bound = xn.copy(), np.abs(xn)
    h = rot // 2
    if h:
        ang = as_f64(positions)[:, None, None] * base ** (-np.arange(h) / h)
        a, b = xn[..., :h], xn[..., h:rot]
        y[..., :h] = a * np.cos(ang) - b * np.sin(ang)
        y[..., h:rot] = b * np.cos(ang) + a * np.sin(ang)
        bound[..., :h] = bound[..., h:rot] = np.abs(a) + np.abs(b)
    return y, bound


def _attend(q, k, v, scale, seen):
    """q [n, d], k, v [m, d], seen [n, m] bool -> (o, a) [n, d]; rows that see nothing are zero."""
    s = np.where(seen, (q @ k.T) * scale, -np.inf)
    top = s.max(-1, keepdims=True, initial=-1e300)
    p = np.exp(s - top)
    l = p.sum(-1, keepdims=True)
    p = p / np.where(l > 0, l, 1.0)
    vv = np.where(seen.any(0)[:, None], v, 0.0)  # an unseen NaN weighs nothing
    return p @ vv, p @ np.abs(vv)


def prompt_attention(q, k, v, seqlens, scale=None):
    """q [T, Hq, d], k, v [T, Hkv, d], packed -> (o, a) [T, Hq, d]."""
    q, k, v = as_f64(q), as_f64(k), as_f64(v)
    T, Hq, d = q.shape
    G = Hq // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    o, a = np.zeros((T, Hq, d)), np.zeros((T, Hq, d))
    t0 = 0
    for n in seqlens:
        causal = np.tri(n, dtype=bool)
        for h in range(Hq):
            r = slice(t0, t0 + n)
            if n:
                o[r, h], a[r, h] = _attend(q[r, h], k[r, h // G], v[r, h // G], scale, causal)
        t0 += n
    return o, a


def decode_attention(q, k_cache, v_cache, table, lens, prefix_pages=None, prefix_len=0, scale=None):
    """q [B, Hq, d]; cache [pages, Hkv, page, d]; table [B, m]; lens [B] -> (o, a) [B, Hq, d]."""
    q, k_cache, v_cache = as_f64(q), as_f64(k_cache), as_f64(v_cache)
    B, Hq, d = q.shape
    page = k_cache.shape[2]
    G = Hq // k_cache.shape[1]
    scale = d ** -0.5 if scale is None else scale
    o, a = np.zeros((B, Hq, d)), np.zeros((B, Hq, d))
    for b in range(B):
        slots = [int(prefix_pages[t // page]) * page + t % page for t in range(prefix_len)]
        slots += [int(table[b][t // page]) * page + t % page for t in range(int(lens[b]))]
        slots = np.array(slots, dtype=np.int64)
        if len(slots) == 0:
            continue
        for h in range(Hq):
            k, v = (c[slots // page, h // G, slots % page] for c in (k_cache, v_cache))
            x, y = _attend(q[b, h][None], k, v, scale, np.ones((1, len(slots)), dtype=bool))
            o[b, h], a[b, h] = x[0], y[0]
    return o, a
