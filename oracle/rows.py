"""Definitions of the operators between the projection's rows and the cache (test
infrastructure only): norm and rotation in float64, attention of packed prompts in float64, the
cache in 4 bits by its own fp32 steps. Plain numpy; nothing is shared with the kernels.
"""

from __future__ import annotations

import numpy as np

GROUP = 32


def norm_rotate(x, weight, positions, frequencies, eps, interleaved):
    """(out, size) float64 of rows x [..., heads, dim] with positions [...]: the result, and
    |y1| + |y2| of the pair that an element is made of (|y| where it is not turned), which
    roundings are relative to. weight None: ones; eps None: no norm."""
    y = np.asarray(x, dtype=np.float64)
    if eps is not None:
        y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps)
        if weight is not None:
            y = y * np.asarray(weight, dtype=np.float64)
    out, size = y.copy(), np.abs(y)
    n = len(frequencies)
    for f in range(n):
        i, j = (2 * f, 2 * f + 1) if interleaved else (f, f + n)
        t = np.asarray(positions, dtype=np.longdouble)[..., None] * np.longdouble(np.float32(frequencies[f]))
        c, s = np.cos(t).astype(np.float64), np.sin(t).astype(np.float64)
        out[..., i] = y[..., i] * c - y[..., j] * s
        out[..., j] = y[..., i] * s + y[..., j] * c
        size[..., i] = size[..., j] = np.abs(y[..., i]) + np.abs(y[..., j])
    return out, size


def prompt_attention(q, k, v, offsets, scale):
    """(out, weight, spread, seen): as in operators.tree_attention, and which tokens are in a sequence."""
    tokens, hq, dim = q.shape
    out, weight = np.zeros(q.shape), np.zeros(q.shape)
    spread, seen = np.zeros((tokens, hq)), np.zeros(tokens, bool)
    for begin, end in zip(offsets, offsets[1:]):
        for i in range(int(begin), int(end)):
            seen[i] = True
            for h in range(hq):
                g = h * k.shape[1] // hq
                kk, vv = (a[begin:i + 1, g].astype(np.float64) for a in (k, v))
                row = q[i, h].astype(np.float64)
                x = scale * (kk @ row)
                p = np.exp(x - x.max())
                p /= p.sum()
                out[i, h] = p @ vv
                weight[i, h] = p @ np.abs(vv)
                spread[i, h] = abs(scale) * (np.abs(kk) @ np.abs(row)).max()
    return out, weight, spread, seen


def q4_codes(x):
    """(codes uint8 [..., dim], scale and low fp16 [..., dim / 32]) of rows of numbers, step by step in fp32."""
    x = np.asarray(x, dtype=np.float32)
    x = np.where(np.isnan(x), np.float32(0), x)
    x = np.clip(x, np.float32(-65408), np.float32(65408)).reshape(*x.shape[:-1], -1, GROUP)
    low, high = x.min(-1), x.max(-1)
    scale = ((high - low) / np.float32(15)).astype(np.float16)
    low = low.astype(np.float16) + np.float16(0)  # no -0
    s, m = scale.astype(np.float32)[..., None], low.astype(np.float32)[..., None]
    steps = (x - m) / np.where(s > 0, s, np.float32(1))
    assert steps.dtype == np.float32
    codes = np.where(s > 0, np.clip(np.rint(steps), 0, 15), 0).astype(np.uint8)
    return codes.reshape(*codes.shape[:-2], -1), scale, low


def q4_pack(x):
    """Rows of bytes uint8 [..., 5 dim / 8] of rows of numbers."""
    codes, scale, low = q4_codes(x)
    rows = []
    for c, s, m in zip(codes.reshape(-1, codes.shape[-1]), scale.reshape(-1, scale.shape[-1]), low.reshape(-1, low.shape[-1])):
        words = []
        for w in range(0, len(c), 8):
            word = 0
            for i in range(4):
                word |= int(c[w + 2 * i]) << (4 * i) | int(c[w + 2 * i + 1]) << (16 + 4 * i)
            words.append(word)
        pairs = np.stack([s, m], -1).reshape(-1)
        rows.append(np.concatenate([np.array(words, "<u4").view(np.uint8), pairs.view(np.uint8)]))
    return np.array(rows).reshape(*codes.shape[:-1], -1)


def q4_unpack(rows):
    """float64 [..., dim]: code * scale + low of rows of bytes, not rounded."""
    rows = np.ascontiguousarray(rows)
    dim = rows.shape[-1] * 8 // 5
    words = np.ascontiguousarray(rows[..., : dim // 2]).view("<u4")
    codes = np.zeros((*rows.shape[:-1], dim))
    for n in range(8):
        codes[..., n::8] = (words >> np.uint32(16 * (n % 2) + 4 * (n // 2))) & np.uint32(15)
    pairs = np.ascontiguousarray(rows[..., dim // 2:]).view(np.float16).astype(np.float64)
    scale, low = (np.repeat(pairs[..., i::2], GROUP, -1) for i in range(2))
    return codes * scale + low


def round_to(x, dt):
    """float64 values rounded to f32, f16 or bf16 (the latter by way of fp32), as float64."""
    if dt == "f16":
        return x.astype(np.float16).astype(np.float64)
    f = x.astype(np.float32)
    if dt == "bf16":
        u = f.view(np.uint32).astype(np.uint64)
        u = (u + 0x7FFF + ((u >> np.uint64(16)) & np.uint64(1))) & np.uint64(0xFFFF0000)
        f = u.astype(np.uint32).view(np.float32)
    return f.astype(np.float64)


def cache_append_q4(k, v, k_cache, v_cache, table, lengths, nodes=None, counts=None):
    """The caches (bytes) after the append; rows go where operators.cache_append puts them."""
    caches = [k_cache.copy(), v_cache.copy()]
    batch, tokens = k.shape[:2]
    pages, page = k_cache.shape[:2]
    for b in range(batch):
        for j in range(tokens if counts is None else min(int(counts[b]), tokens)):
            t = j if nodes is None else int(nodes[b, j])
            pos = int(lengths[b]) + j
            if not (0 <= t < tokens and 0 <= pos < table.shape[1] * page and 0 <= table[b, pos // page] < pages):
                continue
            for cache, rows in zip(caches, (k, v)):
                cache[table[b, pos // page], pos % page] = q4_pack(rows[b, t])
    return caches


def cache_read_q4(k_cache, v_cache, table, lengths, tokens, first, dt):
    """float64 [batch][tokens][heads][dim] twice: the values in type dt, zeros where there is no row."""
    batch, heads = table.shape[0], k_cache.shape[2]
    pages, page = k_cache.shape[:2]
    outs = []
    for cache in (k_cache, v_cache):
        out = np.zeros((batch, tokens, heads, cache.shape[3] * 8 // 5))
        for b in range(batch):
            for j in range(tokens):
                pos = j + (0 if first is None else int(first[b]))
                if 0 <= pos < min(int(lengths[b]), table.shape[1] * page) and 0 <= table[b, pos // page] < pages:
                    out[b, j] = round_to(q4_unpack(cache[table[b, pos // page], pos % page]), dt)
        outs.append(out)
    return outs
