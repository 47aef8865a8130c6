"""Float64 oracle of the paged key-value cache: append, tree attention, commit.

Plain numpy loops from the definitions in include/spec_tree.h, sharing no code
with the CUDA path.  A cache is a pair of arrays [layers][pages][page_size]
[heads][dim], a page table [B][max_pages] and committed lengths [B].  Test
infrastructure only.
"""
from __future__ import annotations

import numpy as np


def sees(parent, n: int):
    """The nodes that node n sees: its ancestors and itself (parent None: every node up to n)."""
    if parent is None:
        return list(range(n + 1))
    out, at = [], n
    while at >= 0:
        out.append(at)
        at = int(parent[at])
    return sorted(out)


def place(table_row, slot: int, page_size: int):
    return int(table_row[slot // page_size]), slot % page_size


def gather(pool, table_row, slots):
    """[len(slots)][heads][dim] float64 of one layer's pool [pages][page_size][heads][dim]."""
    size = pool.shape[1]
    out = np.empty((len(slots),) + pool.shape[2:], np.float64)
    for i, s in enumerate(slots):
        g, o = place(table_row, s, size)
        out[i] = pool[g, o]
    return out


def attend(q, k_pool, v_pool, table, seq_len, parents, counts, begin: int, scale: float):
    """Outputs [B][N][Hq][D], and what their error bounds are made of: the weighted absolute values
    sum p |v| [B][N][Hq][D], the largest sum |q k| scale [B][N][Hq], and sum |v| [B][N][Hq][D]."""
    B, N, Hq, D = q.shape
    Hkv = k_pool.shape[2]
    out, mean_abs, sum_abs = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
    score_abs = np.zeros(q.shape[:3])
    for b in range(B):
        length = int(seq_len[b])
        parent = None if parents is None else parents[b]
        upto = length + min(int(counts[b]), begin + N)
        k, v = gather(k_pool, table[b], range(upto)), gather(v_pool, table[b], range(upto))
        for i in range(N):
            n = begin + i
            if n >= counts[b]:
                continue
            seen = list(range(length)) + [length + a for a in sees(parent, n)]
            for h in range(Hq):
                kk, vv = k[seen, h // (Hq // Hkv)], v[seen, h // (Hq // Hkv)]
                with np.errstate(invalid="ignore", over="ignore"):
                    s = kk @ q[b, i, h] * scale
                    top = s.max()
                    if top == -np.inf:
                        continue
                    w = np.exp(s - top)
                    p = w / w.sum()
                    out[b, i, h] = p @ vv
                    mean_abs[b, i, h] = p @ np.abs(vv)
                    sum_abs[b, i, h] = np.abs(vv).sum(0)
                    score_abs[b, i, h] = (np.abs(kk[w > 0]) @ np.abs(q[b, i, h])).max(initial=0.0) * abs(scale)
    return out, mean_abs, score_abs, sum_abs


def turn(x, weight, eps: float, row, rot_dim: int, interleaved: bool):
    """One head vector: RMS norm (weight None: none) and rotation by a table row (None: none)."""
    x = np.array(x, np.float64)
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x) + eps) * weight
    if row is None:
        return x
    y, half = x.copy(), rot_dim // 2
    for j in range(half):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        c, s = float(row[j]), float(row[half + j])
        y[a], y[b] = x[a] * c - x[b] * s, x[a] * s + x[b] * c
    return y


def append(q, k, v, k_pool, v_pool, table, seq_len, depths, counts, begin, rope, rot_dim, interleaved, qw, kw, eps):
    """(q_out, k_pool, v_pool) of one layer, float64; the pools are copies."""
    k_pool, v_pool, q_out = k_pool.astype(np.float64), v_pool.astype(np.float64), np.zeros(q.shape)
    for b in range(q.shape[0]):
        for i in range(q.shape[1]):
            n = begin + i
            if n >= counts[b]:
                continue
            depth = n if depths is None else int(depths[b][n])
            row = rope[int(seq_len[b]) + depth] if rot_dim else None
            g, o = place(table[b], int(seq_len[b]) + n, k_pool.shape[1])
            for h in range(q.shape[2]):
                q_out[b, i, h] = turn(q[b, i, h], qw, eps, row, rot_dim, interleaved)
            for h in range(k.shape[2]):
                k_pool[g, o, h] = turn(k[b, i, h], kw, eps, row, rot_dim, interleaved)
                v_pool[g, o, h] = v[b, i, h]
    return q_out, k_pool, v_pool


def commit(k_pool, v_pool, table, seq_len, accept_len, out_node):
    """(k_pool, v_pool, new_len) over all layers [layers][pages][page_size][heads][dim]; the pools are copies."""
    k_pool, v_pool, new_len = k_pool.copy(), v_pool.copy(), []
    for b in range(len(seq_len)):
        size, length, a = k_pool.shape[2], int(seq_len[b]), int(accept_len[b])
        for pool in (k_pool, v_pool):
            held = [pool[(slice(None),) + place(table[b], length + int(out_node[b][j]), size)].copy() for j in range(a)]
            for j in range(a):
                pool[(slice(None),) + place(table[b], length + j + 1, size)] = held[j]
        new_len.append(length + 1 + a)
    return k_pool, v_pool, np.array(new_len, np.int32)
