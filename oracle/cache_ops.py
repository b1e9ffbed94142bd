"""Float64 oracle of the cache-maintenance operators: attention of a tree of drafted tokens over a
paged cache, commit of the accepted nodes, accumulated attention mass and eviction by it. Written
from the formulas, one sequence and KV head at a time."""

from __future__ import annotations

import numpy as np


def used_nodes(parents) -> np.ndarray:
    """Nodes that take part: a parent of -1, or an earlier node that takes part."""
    used = np.zeros(len(parents), dtype=bool)
    for i, p in enumerate(parents):
        used[i] = p == -1 or (0 <= p < i and used[p])
    return used


def ancestors(parents) -> list:
    """Per node the list of its ancestors and itself, root first (empty: unused)."""
    used, out = used_nodes(parents), []
    for i, p in enumerate(parents):
        out.append(([] if p == -1 else list(out[p])) + [i] if used[i] else [])
    return out


def row(cache, table, pos, h, page_size):
    """Row of logical position ``pos``, or None on an unusable page or position."""
    if pos < 0 or pos >= len(table) * page_size:
        return None
    page = table[pos // page_size]
    if page < 0 or page >= cache.shape[0]:
        return None
    return cache[page, pos % page_size, h]


def attend(q, k_cache, v_cache, table, positions, h, scale):
    """(output, weights, sum of weight * |v|) of one query over a list of positions; unusable ones
    are left out (weight 0)."""
    ps, d = k_cache.shape[1], q.shape[0]
    w = np.zeros(len(positions))
    rows = [(j, p) for j, p in enumerate(positions) if row(k_cache, table, p, h, ps) is not None]
    if not rows:
        return np.zeros(d), w, np.zeros(d)
    k = np.stack([row(k_cache, table, p, h, ps) for _, p in rows])
    v = np.stack([row(v_cache, table, p, h, ps) for _, p in rows])
    x = k @ q * scale
    e = np.exp(x - x.max())
    e /= e.sum()
    w[[j for j, _ in rows]] = e
    return e @ v, w, e @ np.abs(v)


def tree_positions(parents, i, length, window=-1, idx=None):
    """Positions node ``i`` sees (context, then itself and its ancestors)."""
    anc = ancestors(parents)
    if not anc[i]:
        return []
    depth = len(anc[i]) - 1
    if idx is not None:
        ctx = [int(t) for t in idx]
    else:
        lo = max(0, length + depth - window + 1) if window > 0 else 0
        ctx = list(range(lo, length))
    keep = [a for a in anc[i] if window <= 0 or len(anc[a]) - 1 > depth - window]
    return ctx + [length + a for a in keep]


def tree_attend(q, k_cache, v_cache, block_table, seq_lens, parents, scale, window=-1, idx=None,
                count=None):
    """(output, sum of weight * |v|), both ``[batch, n, h_q, d]``; ``idx`` ``[batch, h_kv, B]``."""
    batch, n, h_q, d = q.shape
    g = h_q // k_cache.shape[2]
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(batch):
        for hq in range(h_q):
            h = hq // g
            sel = None if idx is None else idx[b, h, :count[b, h]]
            for i in range(n):
                pos = tree_positions(parents[b], i, int(seq_lens[b]), window, sel)
                out[b, i, hq], _, mag[b, i, hq] = attend(q[b, i, hq], k_cache, v_cache,
                                                         block_table[b], pos, h, scale)
    return out, mag


def mass_step(q, k_cache, v_cache, block_table, seq_lens, scale, mass, window=-1, idx=None,
              count=None):
    """One decode step's (output, mass + weights): ``mass`` ``[batch, h_kv, capacity]``."""
    batch, h_q, d = q.shape
    h_kv = k_cache.shape[2]
    out, mass = np.zeros(q.shape), mass.astype(np.float64).copy()
    for b in range(batch):
        for hq in range(h_q):
            h = hq // (h_q // h_kv)
            if idx is not None:
                pos = [int(t) for t in idx[b, h, :count[b, h]]]
            else:
                lo = max(0, int(seq_lens[b]) - window) if window > 0 else 0
                pos = list(range(lo, int(seq_lens[b])))
            out[b, hq], w, _ = attend(q[b, hq], k_cache, v_cache, block_table[b], pos, h, scale)
            for p, x in zip(pos, w):
                if x:
                    mass[b, h, p] += x
    return out, mass


def kept_positions(mass, length, keep, recent) -> np.ndarray:
    """Ascending kept positions of one (sequence, KV head); NaN counts as the largest value, ties
    go to the lower position."""
    if length <= keep:
        return np.arange(length)
    m = np.asarray(mass[:length - recent], dtype=np.float64)
    order = sorted(range(len(m)), key=lambda t: (0 if np.isnan(m[t]) else 1,
                                                 0.0 if np.isnan(m[t]) else -m[t], t))
    return np.array(sorted(order[:keep - recent]) + list(range(length - recent, length)))
