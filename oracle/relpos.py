"""The relative position bias and its gradient in 64 bits, buckets by whole numbers."""
from __future__ import annotations

import numpy as np


def borders(buckets, max_distance, both):
    """The smallest distance of each bucket of a direction: e + k begins at the first n with
    n^L e^k >= max_distance^k e^L, L the buckets from e on."""
    half = buckets // 2 if both else buckets
    e = half // 2
    L = half - e
    out = list(range(e + 1))[:half]
    for k in range(1, L):
        lo, hi = e, max_distance
        while lo < hi:
            n = (lo + hi) // 2
            if n ** L * e ** k >= max_distance ** k * e ** L:
                hi = n
            else:
                lo = n + 1
        out.append(lo)
    return out


def bucket(d, buckets, max_distance, both):
    d = np.asarray(d, dtype=np.int64)
    first = np.array(borders(buckets, max_distance, both), dtype=np.int64)
    dist = np.abs(d) if both else np.maximum(-d, 0)
    b = np.searchsorted(first, dist, side="right") - 1
    return b + (buckets // 2) * (d > 0) if both else b


def _which(starts, q, k, buckets, max_distance, both):
    i, j = np.arange(q)[:, None], np.arange(k)[None]
    return [bucket(j - i - int(s), buckets, max_distance, both) for s in starts]


def bias(table, starts, q, k, max_distance, both, scale=1.0, add=None):
    """(batch, heads, q, k); starts: one of each sequence."""
    table = np.asarray(table, dtype=np.float64)
    out = np.stack([np.moveaxis(table[w], 2, 0) * scale for w in _which(starts, q, k, len(table), max_distance, both)])
    return out if add is None else out + add


def grad(dy, starts, buckets, max_distance, both, scale=1.0, old=None):
    """(buckets, heads) and the sums of the terms' sizes that its error is measured by."""
    dy = np.asarray(dy, dtype=np.float64)
    batch, heads, q, k = dy.shape
    total, size = np.zeros((buckets, heads)), np.zeros((buckets, heads))
    for n, w in enumerate(_which(starts, q, k, buckets, max_distance, both)):
        for h in range(heads):
            total[:, h] += np.bincount(w.ravel(), dy[n, h].ravel(), buckets)
            size[:, h] += np.bincount(w.ravel(), np.abs(dy[n, h]).ravel(), buckets)
    total, size = total * scale, size * abs(scale)
    return (total, size) if old is None else (total + old, size + np.abs(old))
