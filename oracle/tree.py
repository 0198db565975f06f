"""Speculative steps over the paged cache in 64 bits: the append of drafted trees, their
attention, the verification of the drafts and the move of the accepted tokens.

The attention forward ("unsloth: compare main...flex-moe-qwen3" · flex_gemma4_moe.py: norm,
rotary, paged write, attention) for several tokens a row that form a tree; verification is
speculative sampling against a draft distribution, sibling after sibling, with the residual
distribution kept normalised.
"""
from __future__ import annotations

import numpy as np

from .norm_rope import rms_norm, rope


def depths(parents):
    """Depth of every node of one row; a parent that is not before its node counts as none."""
    out = []
    for i, p in enumerate(parents):
        out.append(out[p] + 1 if 0 <= p < i else 0)
    return out


def ancestors(parents):
    """bool [n][n]: node t sees node s (its path to the root, itself included)."""
    n = len(parents)
    m = np.eye(n, dtype=bool)
    for i, p in enumerate(parents):
        if 0 <= p < i:
            m[i] |= m[p]
    return m


def rows_of(row_start, parents):
    """(row, first node, parents) of every row."""
    for b in range(len(row_start) - 1):
        n0, n1 = int(row_start[b]), int(row_start[b + 1])
        yield b, n0, [int(p) for p in parents[n0:n1]]


def cache_row(table, slot, pos, page_size):
    return int(table[slot][pos // page_size]) * page_size + pos % page_size


def tree_append(q, k, v, gamma_q, gamma_k, slots, ctx, row_start, parents, theta, eps, rotary_dims,
                v_norm, table, page_size, k_cache, v_cache):
    """Rotated q [N][Hq][D]; writes k_cache and v_cache (float64 [Hkv][rows][D]). v None: the
    raw k."""
    D = q.shape[2]
    v = k if v is None else v
    out = np.array(q)
    for b, n0, par in rows_of(row_start, parents):
        for i, d in enumerate(depths(par)):
            n = n0 + i
            pos = int(ctx[b]) + d
            x, y = q[n], k[n]
            if gamma_q is not None:
                x, y = rms_norm(x, gamma_q, eps), rms_norm(y, gamma_k, eps)
            out[n] = rope(x, pos, theta, rotary_dims)
            r = cache_row(table, slots[b], int(ctx[b]) + i, page_size)
            k_cache[:, r] = rope(y, pos, theta, rotary_dims)
            v_cache[:, r] = rms_norm(v[n], np.ones(D), eps) if v_norm else v[n]
    return out


def tree_attention(q, k_cache, v_cache, table, slots, ctx, row_start, parents, window, scale,
                   page_size, weight_of=None):
    """out [N][Hq][D]; nodes of slot 0 and of no row give zeros. weight_of: also returns
    sum_j p_j |v_j| (how far roundings of the weights can move an output)."""
    N, Hq, D = q.shape
    Hkv = k_cache.shape[0]
    G = Hq // Hkv
    out, mass = np.zeros((N, Hq, D)), np.zeros((N, Hq, D))
    for b, n0, par in rows_of(row_start, parents):
        n, c, slot = len(par), int(ctx[b]), int(slots[b])
        if slot == 0 or n == 0:
            continue
        depth = np.array(depths(par))
        keep = np.concatenate([np.ones((n, c), bool), ancestors(par)], 1)
        if window > 0:
            pos = np.concatenate([np.arange(c), c + depth])
            keep &= (c + depth)[:, None] - pos[None] < window
        rows = [cache_row(table, slot, j, page_size) if keep[:, j].any() else 0
                for j in range(c + n)]
        for h in range(Hq):
            K, V = k_cache[h // G][rows], v_cache[h // G][rows]
            for t in range(n):
                j = keep[t]
                s = scale * (K[j] @ q[n0 + t, h])
                p = np.exp(s - s.max())
                p /= p.sum()
                out[n0 + t, h] = p @ V[j]
                mass[n0 + t, h] = p @ np.abs(V[j])
    return (out, mass) if weight_of else out


def _clean(p):
    return np.clip(np.nan_to_num(np.asarray(p, np.float64), nan=0.0), 0.0, 1.0)


def tree_verify(target, draft, tokens, row_start, parents, u_accept, u_pick, path_cols):
    """(accepted [B], path [B][path_cols], next [B]). A node's children are tried in order; the
    distribution left after a refusal is kept normalised."""
    B = len(row_start) - 1
    accepted, path, nxt = np.zeros(B, int), np.full((B, path_cols), -1), np.full(B, -1)
    V = target.shape[1]
    for b, n0, par in rows_of(row_start, parents):
        if not par:
            continue
        cur, walk = 0, [0]
        dist = _clean(target[n0])
        for i in range(1, len(par)):
            if par[i] != cur or not 0 <= tokens[n0 + i] < V:
                continue
            x = int(tokens[n0 + i])
            q = _clean(draft[n0 + cur]) if draft is not None else None
            if float(u_accept[n0 + i]) * (1.0 if q is None else q[x]) < dist[x]:
                cur = i
                walk.append(i)
                dist = _clean(target[n0 + i])
                continue
            if q is None:
                left = 1.0 - dist[x]
                dist = dist.copy()
                dist[x] = 0.0
                dist = dist / left if left > 0 else dist
            else:
                dist = np.maximum(dist - q, 0.0)
                dist = dist / dist.sum() if dist.sum() > 0 else dist
        if dist.sum() == 0:
            dist = _clean(target[n0 + cur])
        c = np.cumsum(dist)
        if c[-1] > 0:
            nxt[b] = int(np.argmax(c > float(u_pick[b]) * c[-1]))
        accepted[b] = len(walk) - 1
        path[b, :len(walk)] = walk
    return accepted, path, nxt


def keep_path(cache, table, slots, ctx, accepted, path, page_size):
    """Moves the accepted tokens of every row inside `cache` [heads][rows][...]."""
    for b in range(len(accepted)):
        if slots[b] == 0:
            continue
        for t in range(1, int(accepted[b]) + 1):
            src = cache_row(table, slots[b], int(ctx[b]) + int(path[b][t]), page_size)
            dst = cache_row(table, slots[b], int(ctx[b]) + t, page_size)
            cache[:, dst] = cache[:, src]
