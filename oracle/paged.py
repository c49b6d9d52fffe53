"""Oracle of the paged serving operators: page plan, rotation and store, single-token attention, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Each function is the operator's definition, one
request or token at a time, on numpy arrays; e4m3 inputs come decoded.
"""
from __future__ import annotations

import numpy as np


def paged_plan(cached, new, table, free, cursor, page, max_tokens):
    """(table, seq_lens, cu_tokens, positions, slots, cursor, capacity_met) of a step; inputs are not changed.

    Requests take pages in order; a token without a page (pool or table exhausted) has slot -1.
    """
    table = np.array(table, dtype=np.int32)
    width = table.shape[1]
    lens, cu, positions, slots = [], [0], [], []
    taken, met = int(cursor), False
    for b, (c, n) in enumerate(zip(cached, new)):
        c, n = max(0, int(c)), max(0, int(n))
        for p in range(min(-(-c // page), width), min(-(-(c + n) // page), width)):
            table[b, p] = free[taken] if taken < len(free) else -1
            met |= taken >= len(free)
            taken += 1
        for pos in range(c, c + n):
            positions.append(pos)
            p = pos // page
            if p < width and table[b, p] >= 0:
                slots.append(int(table[b, p]) * page + pos % page)
            else:
                slots.append(-1)
                met = True
        lens.append(min(c + n, width * page))
        met |= c + n > width * page
        cu.append(cu[-1] + n)
    met |= cu[-1] > max_tokens
    tail = max(0, max_tokens - cu[-1])
    positions = np.array((positions + [0] * tail)[:max_tokens], dtype=np.int32)
    slots = np.array((slots + [-1] * tail)[:max_tokens], dtype=np.int64)
    return (table, np.array(lens, dtype=np.int32), np.array(cu, dtype=np.int32), positions, slots,
            max(min(taken, len(free)), int(cursor)), met)


def rope_rotate(x, positions, inv_freq, axis_pairs, offset=0, interleaved=False):
    """Rotate x [N, heads, D] (float64): pair i of token n by positions[axis(i)][n] * inv_freq[i]."""
    y = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    axis = np.repeat(np.arange(len(axis_pairs)), axis_pairs)
    for i in range(half):
        angle = np.asarray(positions, dtype=np.float64)[axis[i]] * np.float64(inv_freq[i])
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        d0, d1 = (offset + 2 * i, offset + 2 * i + 1) if interleaved else (offset + i, offset + i + half)
        a, b = np.array(y[..., d0]), np.array(y[..., d1])
        y[..., d0], y[..., d1] = a * c - b * s, a * s + b * c
    return y


def decode_attention(q, k, v, scale):
    """One query row q [D_qk] over keys k [n, D_qk] and values v [n, D_v]: (out, lse, weights)."""
    if len(k) == 0:
        return np.zeros(v.shape[1]), -np.inf, np.zeros(0)
    x = k @ q * scale
    m = x.max()
    w = np.exp(x - m)
    total = w.sum()
    return w @ v / total, m + np.log(total), w / total
