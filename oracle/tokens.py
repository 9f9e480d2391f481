"""Rows sorted by expert, the weighted way back and its gradient, in float64.

The layout (rows of each slot, padded blocks) is oracle.moe's dispatch layout.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""

import numpy as np

GROUP = 128


def layout(topk_ids, G):
    """(row_of_slot int32 T x topk, m_offsets int32[G+1], counts): slot order inside an expert."""
    ids = np.asarray(topk_ids, np.int64)
    rows = np.full(ids.size, -1, np.int64)
    off = np.zeros(G + 1, np.int64)
    counts = np.zeros(G, np.int64)
    flat = ids.reshape(-1)
    for e in range(G):
        slots = np.nonzero(flat == e)[0]
        counts[e] = slots.size
        rows[slots] = off[e] + np.arange(slots.size)
        off[e + 1] = off[e] + (slots.size + GROUP - 1) // GROUP * GROUP
    return rows.reshape(ids.shape).astype(np.int32), off.astype(np.int32), counts


def permute(x, topk_ids, G):
    """(xp rows [0, m_offsets[G]), m_offsets, row_of_slot); x of any dtype, copied bit for bit."""
    rows, off, _ = layout(topk_ids, G)
    xp = np.zeros((int(off[-1]), x.shape[1]), x.dtype)
    t, j = np.nonzero(rows >= 0)
    xp[rows[t, j]] = x[t]
    return xp, off, rows


def combine(c, rows, weights=None):
    """(y, sum of the terms' magnitudes), float64; rows outside c contribute nothing."""
    c, rows = np.asarray(c, np.float64), np.asarray(rows)
    T, topk = rows.shape
    y, mag = np.zeros((T, c.shape[1])), np.zeros((T, c.shape[1]))
    for t in range(T):
        for j in range(topk):
            if 0 <= rows[t, j] < c.shape[0]:
                term = c[rows[t, j]] * (1.0 if weights is None else float(weights[t, j]))
                y[t] += term
                mag[t] += np.abs(term)
    return y, mag


def combine_bwd(dy, c, rows, weights, m_offsets):
    """(dc with NaN where nothing is written, dw, sum of dw's terms' magnitudes), float64."""
    dy, c, rows = np.asarray(dy, np.float64), np.asarray(c, np.float64), np.asarray(rows)
    T, topk = rows.shape
    M = c.shape[0]
    dc = np.full(c.shape, np.nan)
    dw, mag = np.zeros((T, topk)), np.zeros((T, topk))
    off = np.clip(np.asarray(m_offsets, np.int64), 0, M)
    for e in range(len(off) - 1):
        inside = rows[(rows >= off[e]) & (rows < off[e + 1])]
        first = int(inside.max()) + 1 if inside.size else int(off[e])
        dc[first:int(off[e + 1])] = 0.0
    for t in range(T):
        for j in range(topk):
            r = rows[t, j]
            if 0 <= r < M:
                dc[r] = dy[t] * (1.0 if weights is None else float(weights[t, j]))
                dw[t, j] = float(dy[t] @ c[r])
                mag[t, j] = float(np.abs(dy[t]) @ np.abs(c[r]))
    return dc, dw, mag
