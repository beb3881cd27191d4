"""Rotary positions, the append to a paged MXFP8 cache and attention over it, in
64 bits from their definitions (numpy, no code shared with the library).

A cache is a tuple (k codes, k scales, v codes, v scales) of uint8 arrays
[pages][kv_heads][page][dim] and [..][dim / 32].
"""

import math

import numpy as np

from . import mx


def frequencies(rot, base, scaling="none", factor=1.0, orig_len=0):
    """(angle per position of every pair, factor on cos and sin)."""
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2.0))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        def channel(turns):
            """The channel that turns this often over the original length."""
            return rot * math.log(orig_len / (2 * math.pi * turns)) / (2 * math.log(base))
        lo, hi = max(math.floor(channel(32)), 0), min(math.ceil(channel(1)), rot - 1)
        r = np.clip((i - lo) / max(hi - lo, 1e-3), 0, 1)
        return f * (1 - r) + f / factor * r, 1.0 + 0.1 * math.log(factor)
    if scaling == "bands":
        s = np.clip((orig_len * f / (2 * math.pi) - 1) / 3, 0, 1)
        return s * f + (1 - s) * f / factor, 1.0
    return f, 1.0


def rope_table(rows, rot, base, scaling="none", factor=1.0, orig_len=0):
    f, m = frequencies(rot, base, scaling, factor, orig_len)
    a = np.arange(rows, dtype=np.float64)[:, None] * f
    return np.stack([np.cos(a) * m, np.sin(a) * m], -1)


def rotate(x, pos, table, layout="half", inverse=False):
    """x [tokens][heads][dim] turned by table rows [rot / 2][2] of pos, in x's own precision."""
    x = np.asarray(x)
    table = np.asarray(table, dtype=x.dtype)
    half = table.shape[1]
    c, s = table[pos][:, None, :, 0], table[pos][:, None, :, 1]
    if inverse:
        s = -s
    y = x.copy()
    first = slice(0, half) if layout == "half" else slice(0, 2 * half, 2)
    second = slice(half, 2 * half) if layout == "half" else slice(1, 2 * half, 2)
    a, b = x[..., first], x[..., second]
    y[..., first] = a * c - b * s
    y[..., second] = b * c + a * s
    return y


def append(cache, k, v, slots):
    """Stores FP32 keys and values [tokens][kv_heads][dim]; slots outside the cache are skipped."""
    pages, heads, page, dim = cache[0].shape
    for x, codes, scales in ((k, cache[0], cache[1]), (v, cache[2], cache[3])):
        q, s = mx.quantize_rowwise(np.asarray(x, dtype=np.float32).reshape(-1, dim), "e4m3", "ceil")
        q, s = q.reshape(len(slots), heads, dim), s.reshape(len(slots), heads, dim // 32)
        for t, slot in enumerate(slots):
            if 0 <= slot < pages * page:
                codes[slot // page, :, slot % page] = q[t]
                scales[slot // page, :, slot % page] = s[t]


def attention(q, cache, page_table, cu, lens, window=0, scale=None):
    """(out, lse, weighted sum of |v|, largest sum of |q k| over the keys, its keys) of every query and head.

    The last three bound what rounding the weights and the products can change.  Queries that see
    a token of a page out of range, or past the table, are NaN."""
    pages, hk, page, dim = cache[0].shape
    tokens, heads, _ = q.shape
    group = heads // hk
    c = dim ** -0.5 if scale is None else scale
    val = [mx.dequantize_exact(cache[n].reshape(-1, dim), cache[n + 1].reshape(-1, dim // 32), "e4m3")
           .reshape(pages, hk, page, dim) if pages else np.zeros((0, hk, page, dim)) for n in (0, 2)]
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    lse, big, seen = np.full((tokens, heads), -np.inf), np.zeros((tokens, heads)), np.zeros((tokens, heads), dtype=int)
    for r in range(len(lens)):
        m, n = int(cu[r + 1] - cu[r]), int(lens[r])
        for i in range(m):
            p = n - m + i
            keys = np.arange(max(0, p - window + 1) if window else 0, p + 1)
            if not len(keys):
                continue
            col = keys // page
            ok = col < page_table.shape[1]
            ids = page_table[r, np.where(ok, col, 0)] if page_table.shape[1] else np.zeros(len(keys), int)
            ok &= (ids >= 0) & (ids < pages)
            t = cu[r] + i
            if not ok.all():
                out[t], mag[t], lse[t] = np.nan, np.nan, np.nan
                continue
            for h in range(heads):
                k, v = (x[ids, h // group, keys % page] for x in val)
                x = q[t, h].astype(np.float64)
                s = c * (k @ x)
                top = s.max()
                e = np.exp(s - top)
                lse[t, h] = top + np.log(e.sum())
                e /= e.sum()
                out[t, h] = e @ v
                mag[t, h] = e @ np.abs(v)
                big[t, h] = c * (np.abs(k) @ np.abs(x)).max()
                seen[t, h] = len(keys)
    return out, lse, mag, big, seen
