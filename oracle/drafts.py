"""fp64 oracle of a decode step with drafted tokens: rotary positions, the keys
that a node of a tree attends to, and which drafted tokens are kept.

Written from the definitions, a row (a node, a sequence) at a time.
"""
from __future__ import annotations

import numpy as np


def turn(x, positions, inv_freq, magnitude=1.0, interleaved=False):
    """x [rows, heads, dim] with its first 2 len(inv_freq) channels turned, as products with magnitude e^(i t)."""
    y, n = np.array(x, dtype=np.float64), len(inv_freq)
    t = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    z = (y[..., a] + 1j * y[..., b]) * (magnitude * np.exp(1j * t))[:, None]
    y[..., a], y[..., b] = z.real, z.imag
    return y


def line(parents, node):
    """The node and its ancestors, from itself up; None if a parent is not below its node or is less than -1."""
    up = []
    while node != -1:
        up.append(node)
        if not -1 <= parents[node] < node:
            return None
        node = parents[node]
    return up


def keys_of(parents, node, base, window=0):
    """Positions that a node of a tree behind `base` keys attends to, in rising order; None: no valid way up."""
    up = line(parents, node)
    if up is None:
        return None
    position = base + len(up) - 1
    before = range(max(0, position - window + 1) if window else 0, base)
    return np.array(list(before) + sorted(base + x for x in (up[:window] if window else up)), dtype=np.int64)


def attend(q, k, v, scale):
    """One query over the keys it attends to: o, lse, and what error bounds need (oracle.int8.attention)."""
    t = scale * (k @ q)
    w = np.exp(t - t.max())
    return (w @ v / w.sum(), t.max() + np.log(w.sum()), w @ np.abs(v) / w.sum(), abs(scale) * (np.abs(k) @ np.abs(q)).max(),
            np.abs(t).max())


def verify(target, draft, tokens, parents, u, r):
    """One sequence: (kept nodes, next token). target, draft [n, vocab] (draft None: drafts that were chosen)."""
    n, vocab = target.shape
    if n == 0:
        return [], -1
    target = np.asarray(target, np.float64)
    kept, node = [0], 0
    while True:
        w, z, found = np.maximum(target[node], 0), 1.0, -1
        for x in range(node + 1, n):
            if parents[x] != node or not 0 <= tokens[x] < vocab:
                continue
            q = np.zeros(vocab) if draft is None else np.asarray(draft[node], np.float64)
            if draft is None:
                q[tokens[x]] = 1.0
            if u[x] * z * q[tokens[x]] < w[tokens[x]]:
                found = x
                break
            if draft is None:
                z -= w[tokens[x]]
                w[tokens[x]] = 0
            else:
                w = np.maximum(w - z * q, 0)
                z = w.sum()
        if found < 0:
            break
        kept.append(found)
        node = found
    if w.sum() == 0:
        w = np.maximum(target[node], 0)
    total = w.sum()
    if not 0 < total < np.inf:
        return kept, -1
    over = np.nonzero(np.cumsum(w) > r * total)[0]
    return kept, int(over[0]) if len(over) else int(np.nonzero(w)[0][-1])
