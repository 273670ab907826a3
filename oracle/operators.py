"""Float64 definitions of the operators around the projection (test infrastructure
only): tree attention over a paged cache, the cache's append, verification of drafts
from given random numbers, distillation from a teacher's top logits. Plain numpy, one
sequence, head and row at a time; nothing is shared with the kernels.
"""

from __future__ import annotations

import numpy as np


def cached_rows(cache, table_row, length, head):
    """[length][dim] float64 rows of one sequence and head from a cache [pages][slots][heads][dim]."""
    page = cache.shape[1]
    pos = np.arange(length)
    return cache[table_row[pos // page], pos % page, head].astype(np.float64)


def tree_attention(q, k, v, mask, k_cache, v_cache, table, lengths, scale):
    """(out, weight, spread), float64 [batch][nodes][q_heads][dim] twice and [batch][nodes]
    [q_heads]: the output, sum_j p_j |V_j| (what roundings of p are relative to) and the
    largest scale * sum_d |q_d K_jd| (what roundings of the scores are relative to). Only
    the keys that a node sees enter, so values elsewhere have no say."""
    batch, nodes, hq, dim = q.shape
    hkv = k.shape[2]
    out = np.zeros(q.shape)
    weight = np.zeros(q.shape)
    spread = np.zeros(q.shape[:3])
    for b in range(batch):
        for g in range(hkv):
            ck = cached_rows(k_cache, table[b], int(lengths[b]), g)
            cv = cached_rows(v_cache, table[b], int(lengths[b]), g)
            for i in range(nodes):
                seen = [t for t in range(nodes) if (int(mask[b, i]) >> t) & 1]
                kk = np.concatenate([ck, k[b, seen, g].astype(np.float64).reshape(-1, dim)])
                vv = np.concatenate([cv, v[b, seen, g].astype(np.float64).reshape(-1, dim)])
                if len(kk) == 0:
                    continue
                for h in range(g * hq // hkv, (g + 1) * hq // hkv):
                    row = q[b, i, h].astype(np.float64)
                    x = scale * (kk @ row)
                    p = np.exp(x - x.max())
                    p /= p.sum()
                    out[b, i, h] = p @ vv
                    weight[b, i, h] = p @ np.abs(vv)
                    spread[b, i, h] = abs(scale) * (np.abs(kk) @ np.abs(row)).max()
    return out, weight, spread


def cache_append(k, v, k_cache, v_cache, table, lengths, nodes=None, counts=None):
    """The caches after the append (copies), any element type."""
    kc, vc = k_cache.copy(), v_cache.copy()
    batch, tokens = k.shape[:2]
    pages, page = kc.shape[:2]
    for b in range(batch):
        count = tokens if counts is None else max(0, min(tokens, int(counts[b])))
        for j in range(count):
            t = j if nodes is None else int(nodes[b, j])
            pos = int(lengths[b]) + j
            if not 0 <= t < tokens or not 0 <= pos < table.shape[1] * page:
                continue
            to = int(table[b, pos // page])
            if 0 <= to < pages:
                kc[to, pos % page] = k[b, t]
                vc[to, pos % page] = v[b, t]
    return kc, vc


def weights(row, temperature):
    """Float64 weights of a row of logits (not divided by their sum)."""
    x = np.where(np.isnan(row), -np.inf, row.astype(np.float64))
    w = np.zeros(len(x))
    top = x.max()
    if top == -np.inf:
        return w
    if not temperature > 0:
        w[int(np.argmax(x))] = 1.0
    elif top == np.inf:
        w[x == np.inf] = 1.0
    else:
        w = np.exp((x - top) / float(temperature))
    return w


def fraction(u):
    """A random number as it is used: NaN and what is below 0 count as 0."""
    return float(u) if u > 0 else 0.0


def sample(w, u):
    """First place whose running sum is over u times the sum; the last with weight at most."""
    at = np.flatnonzero(w > 0)
    if len(at) == 0:
        return -1
    c, u = np.cumsum(w), fraction(u)
    over = np.flatnonzero(c > u * c[-1])
    return int(min(over[0], at[-1])) if len(over) else int(at[-1])


def verify_tree(logits, tokens, parents, u, temperature=None):
    batch, nodes, _ = logits.shape
    accepted = np.full((batch, nodes), -1, np.int32)
    count, after = np.zeros(batch, np.int32), np.zeros(batch, np.int32)
    for b in range(batch):
        t = 1.0 if temperature is None else temperature[b]
        node, path = 0, []
        while True:
            path.append(node)
            token = sample(weights(logits[b, node], t), u[b, node])
            child = [c for c in range(node + 1, nodes) if parents[b, c] == node and tokens[b, c] == token and token >= 0]
            if not child:
                break
            node = child[0]
        accepted[b, : len(path)] = path
        count[b], after[b] = len(path), token
    return accepted, count, after


def verify_chain(logits, tokens, q, u, temperature=None):
    batch, nodes, vocab = logits.shape
    count, after = np.zeros(batch, np.int32), np.zeros(batch, np.int32)
    for b in range(batch):
        t = 1.0 if temperature is None else temperature[b]
        for j in range(nodes):
            w = weights(logits[b, j], t)
            p = w / w.sum() if w.sum() > 0 else w
            if j + 1 < nodes:
                x = int(tokens[b, j + 1])
                if 0 <= x < vocab and fraction(u[b, j]) * float(q[b, j, x]) < p[x]:
                    continue
                rest = np.maximum(p - q[b, j].astype(np.float64), 0.0)
                p = rest if (rest > 0).any() else p
            count[b], after[b] = j + 1, sample(p, u[b, nodes - 1])
            break
    return count, after


def distill(logits, index, top, weight, temperature):
    """(loss, grad, p, t): float64 loss [rows], gradient and student probabilities
    [rows][vocab], and the teacher's mass at each place [rows][vocab]."""
    rows, vocab = logits.shape
    loss, grad = np.zeros(rows), np.zeros((rows, vocab))
    p, t = np.zeros((rows, vocab)), np.zeros((rows, vocab))
    for r in range(rows):
        x = logits[r].astype(np.float64) / temperature
        lp = x - x.max()
        lp -= np.log(np.exp(lp).sum())
        p[r] = np.exp(lp)
        there = (index[r] >= 0) & (index[r] < vocab)
        if not there.any():
            continue
        at = index[r][there]
        y = top[r][there].astype(np.float64) / temperature
        ly = y - y.max()
        ly -= np.log(np.exp(ly).sum())
        ty = np.exp(ly)
        use = ty > 0
        loss[r] = np.sum(ty[use] * (ly[use] - lp[at[use]]))
        np.add.at(t[r], at, ty)
        if weight is not None and weight[r] != 0:
            grad[r] = weight[r] / temperature * (p[r] - t[r])
    return loss, grad, p, t
