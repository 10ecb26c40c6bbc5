"""Plain numpy references of the verify round's operators beside the MoE layer, in float64.

Written from the definitions in include/verify_ops.h, request by request and row by row; they share no
code with the GPU path.  16-bit inputs are passed as float64 arrays of their values.
"""
from __future__ import annotations

import math

import numpy as np


def round_slots(cached, rows, table, free_pages, page_size, total_rows, parents=None, free_head=0):
    """(row_start, slots, positions, masks or None, counts, table) of a round; `table` is not changed."""
    table = np.array(table, dtype=np.int64)
    B, W = table.shape
    P, N, F = page_size, total_rows, len(free_pages)
    row_start, slots, positions, masks = [], [-1] * N, [0] * N, [0] * N
    start = taken = 0
    for b in range(B):
        c, r = max(int(cached[b]), 0), max(int(rows[b]), 0)
        row_start.append(min(start, N))
        for col in range(min(-(-c // P), W), min(-(-(c + r) // P), W)):
            at = free_head + taken
            table[b, col] = free_pages[at] if 0 <= at < F else -1
            taken += 1
        depth, bits = [], []
        for i in range(r):
            t = start + i
            if parents is None:
                depth.append(i)
            elif i < 64 and t < N:
                up = int(parents[t])
                up = up if 0 <= up < i else -1
                depth.append(depth[up] + 1 if up >= 0 else 0)
                bits.append((1 << i) | (bits[up] if up >= 0 else 0))
            if t >= N:
                continue
            if parents is not None and i >= 64:
                positions[t] = c
                continue
            col, place = divmod(c + i, P)
            page = int(table[b, col]) if col < W else -1
            slots[t] = page * P + place if page >= 0 else -1
            positions[t] = c + depth[i]
            if parents is not None:
                masks[t] = bits[i]
        start += r
    row_start.append(min(start, N))
    m = np.array(masks, dtype=np.uint64).view(np.int64) if parents is not None else None
    return (np.array(row_start, np.int32), np.array(slots, np.int32), np.array(positions, np.int32), m,
            np.array([start, taken], np.int32), table.astype(np.int32))


def norm_rope(x, weight, positions, inv_freq, eps, interleaved):
    """x [T, heads, D] normed (weight None: not) and its first 2 * len(inv_freq) values rotated."""
    x = np.array(x, dtype=np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    y = x.copy()
    half = len(inv_freq)
    for t in range(x.shape[0]):
        for i in range(half):
            angle = float(positions[t]) * float(inv_freq[i])
            c, s = math.cos(angle), math.sin(angle)
            p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            a, b = x[t, :, p], x[t, :, q]
            y[t, :, p] = a * c - b * s
            y[t, :, q] = b * c + a * s
    return y


def tree_attention(q, k_cache, v_cache, table, cached, row_start, masks, max_rows, scale):
    """(out, spread, reach): the rows' attention [T, heads, D] (NaN in rows no request owns), sum_j p_j |v_j|
    per element, and the largest sum_d |q_d k_jd| * scale over the seen tokens per (row, head)."""
    q = np.asarray(q, np.float64)
    T, heads, D = q.shape
    pages, kv_heads, P, _ = k_cache.shape
    group = heads // kv_heads
    out = np.full(q.shape, np.nan)
    spread, reach = np.zeros(q.shape), np.zeros((T, heads))
    W = table.shape[1]
    for b in range(table.shape[0]):
        first, rows = int(row_start[b]), int(row_start[b + 1]) - int(row_start[b])
        c = max(int(cached[b]), 0)
        for i in range(min(rows, max_rows)):
            word = (int(masks[first + i]) & (2 ** 64 - 1)) if masks is not None else (1 << (i + 1)) - 1
            seen = list(range(min(c, W * P))) + [c + j for j in range(min(rows, max_rows, 64)) if (word >> j) & 1]
            where = [(int(table[b, j // P]), j % P) for j in seen if j // P < W]
            where = [(p, o) for p, o in where if 0 <= p < pages]
            if not where:
                out[first + i] = 0
                continue
            pg, of = np.array(where).T
            for h in range(heads):
                k = np.asarray(k_cache[pg, h // group, of], np.float64)
                v = np.asarray(v_cache[pg, h // group, of], np.float64)
                s = scale * (k @ q[first + i, h])
                with np.errstate(invalid="ignore", over="ignore"):
                    e = np.exp(s - s.max())
                    p = e / e.sum()
                    out[first + i, h] = p @ v
                    spread[first + i, h] = p @ np.abs(v)
                    reach[first + i, h] = scale * (np.abs(k) @ np.abs(q[first + i, h])).max()
    return out, spread, reach


def token_logprobs(logits, tokens, top):
    """(logprobs, entropy, top_ids, top_logprobs) of logits [T, V] without NaN and +inf."""
    x = np.asarray(logits, np.float64)
    T, V = x.shape
    lp = np.full(tokens.shape, -np.inf)
    entropy, ids, tlp = np.zeros(T), np.zeros((T, top), np.int32), np.zeros((T, top))
    for t in range(T):
        m = x[t].max()
        order = np.argsort(-x[t], kind="stable")[:top]
        ids[t] = order
        if m == -np.inf:
            tlp[t] = -np.inf
            continue
        e = np.exp(x[t] - m)
        z = m + math.log(e.sum())
        p = e / e.sum()
        some = p > 0
        entropy[t] = -(p[some] * (x[t][some] - z)).sum()
        tlp[t] = x[t][order] - z
        for n, tok in enumerate(tokens[t]):
            if 0 <= tok < V:
                lp[t, n] = x[t, tok] - z
    return lp, entropy, ids, tlp
