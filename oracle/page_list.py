"""Plain 64-bit restatement of the operators over lists of cached chunks -- TEST
INFRASTRUCTURE ONLY.

Attention of new tokens, the weight that chunks gather from them, and eviction by
that weight.  bf16 values are passed as fp64 numbers.  Pinned by
``tests/test_page_list_oracle.py``.
"""
from __future__ import annotations

import numpy as np

__all__ = ["list_rows", "extend_attention", "chunk_weights", "evict_unit"]


def list_rows(pool, staged, idx, slot, cs):
    """Rows [n*cs, 128] of a list's chunks and their positions."""
    rows = [pool[s] if s >= 0 else staged[-1 - s] for s in slot]
    rows = np.concatenate(rows) if rows else np.zeros((0, 128))
    pos = (np.asarray(idx, np.int64)[:, None] * cs + np.arange(cs)).reshape(-1)
    return rows, pos


def extend_attention(q, p0, K, V, pos, scale):
    """q [T, G, 128] at positions p0, p0 + 1, ..: (out [T, G, 128], lse [T, G]) over the rows at positions up
    to each token's own."""
    T, G, D = q.shape
    out, lse = np.zeros((T, G, D)), np.full((T, G), -np.inf)
    for t in range(T):
        see = pos <= p0 + t
        if not see.any():
            continue
        x = q[t] @ K[see].T * scale
        top = x.max(-1, keepdims=True)
        with np.errstate(invalid="ignore"):
            w = np.exp(x - np.where(np.isneginf(top), 0.0, top))
        s = w.sum(-1, keepdims=True)
        some = s[:, 0] != 0
        with np.errstate(invalid="ignore", divide="ignore"):
            out[t] = np.where(some[:, None], (w / s) @ V[see], 0.0)
            lse[t] = np.where(some, np.where(np.isneginf(top), 0.0, top)[:, 0] + np.log(s[:, 0]), -np.inf)
    return out, lse


def chunk_weights(q, p0, lse, K, pos, cs, scale, first=0):
    """Weights [n] that a list's n chunks gather from tokens first .. T-1."""
    n = len(pos) // cs
    w = np.zeros(n)
    for t in range(first, q.shape[0]):
        for h in range(q.shape[1]):
            if np.isneginf(lse[t, h]):
                continue
            p = np.where(pos <= p0 + t, np.exp(K @ q[t, h] * scale - lse[t, h]), 0.0)
            w += p.reshape(n, cs).sum(-1)
    return w


def evict_unit(weight, resident, base, S, n0, n1, keep, first, last):
    """One unit: (resident map after the call, chunks that left, whether slots ran out)."""
    now = np.array(resident, np.int64)
    held = [c for c in range(len(now)) if now[c] >= 0]
    come = [c for c in range(n0, n1) if now[c] < 0]
    cand = [c for c in held if first <= c < n0 - last]
    e = min(max(len(held) + len(come) - keep, 0), len(cand))
    rank = sorted(cand, key=lambda c: (0, 0.0, c) if np.isnan(weight[c]) else (1, float(weight[c]) + 0.0, c))
    gone = sorted(rank[:e])
    for c in gone:
        now[c] = -1
    taken = set(int(s) for s in now if s >= 0)
    free = [s for s in range(base, base + S) if s not in taken]
    for c, s in zip(come, free):
        now[c] = s
    return now, gone, len(come) > len(free)
