"""Embedding lookup, its gradient and counter-based dropout, in 64 bits.

Definitions (e counts the elements of the dropped tensor row by row):

  u(e) = 2^16 h + l, with h the 16-bit half e mod 8 of the four words of
  Philox4x32-10 (low half of the first word first) at key (seed low, seed high) and
  counter (b low, b high, site, step low), b = e div 8, and l the same half at
  (b low, b high | 2^31, site, step low);
  T = floor(p 2^32); e is dropped iff u(e) < T; k = 1 / (1 - T 2^-32).

  dropout  y[e]      = (add[e] or 0) + (dropped(e) ? 0 : x[e] k)
  lookup   out[i, c] = id_i a row and kept ? table[id_i, c] scale k : 0
  grad     G[v, c]   = (G[v, c] or 0) + scale k sum of the kept dy[i, c] with id_i = v

Philox4x32-10 is written from its published definition (Salmon, Moraes, Dror, Shaw,
"Parallel random numbers: as easy as 1, 2, 3", SC'11).
"""
from __future__ import annotations

import numpy as np

_M32 = np.uint64(0xFFFFFFFF)
_32 = np.uint64(32)


def philox4x32_10(counter, key):
    """Four uint64 arrays of 32-bit words and two key words -> four such arrays."""
    c = [np.asarray(x, dtype=np.uint64) for x in counter]
    k0, k1 = int(key[0]), int(key[1])
    for _ in range(10):
        p0, p1 = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(p1 >> _32) ^ c[1] ^ np.uint64(k0), p1 & _M32,
             (p0 >> _32) ^ c[3] ^ np.uint64(k1), p0 & _M32]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c


def threshold(p):
    return int(np.floor(p * 2.0 ** 32))


def keep_scale(p):
    return 1.0 / (1.0 - threshold(p) * 2.0 ** -32)


def numbers(first, n, seed, step, site):
    """u(e) for e in [first, first + n)."""
    b = np.arange(first // 8, (first + n + 7) // 8, dtype=np.uint64)

    def halves(top):
        w = philox4x32_10([b & _M32, (b >> _32) | np.uint64(top), np.full_like(b, site),
                           np.full_like(b, step & 0xFFFFFFFF)], (seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF))
        return np.stack([h for x in w for h in (x & np.uint64(0xFFFF), x >> np.uint64(16))], axis=1).ravel()

    u = halves(0) << np.uint64(16) | halves(1 << 31)
    return u[first % 8:first % 8 + n]


def kept(first, n, p, seed, step, site):
    return numbers(first, n, seed, step, site) >= np.uint64(threshold(p))


def dropout(x, p, seed, step, site, add=None):
    x = np.asarray(x, dtype=np.float64)
    y = np.where(kept(0, x.size, p, seed, step, site).reshape(x.shape), x * keep_scale(p), 0.0)
    return y if add is None else np.asarray(add, dtype=np.float64) + y


def lookup(ids, table, scale=1.0, p=0.0, seed=0, step=0, site=0):
    ids, table = np.asarray(ids).ravel(), np.asarray(table, dtype=np.float64)
    rows, dim = table.shape
    out = np.zeros((ids.size, dim))
    ok = (ids >= 0) & (ids < rows)
    out[ok] = table[ids[ok]] * (scale * keep_scale(p))
    if threshold(p):
        out[~kept(0, out.size, p, seed, step, site).reshape(out.shape)] = 0.0
    return out


def grad(ids, dy, rows, scale=1.0, p=0.0, seed=0, step=0, site=0, old=None):
    """The gradient, and the sum of the absolute values of each element's terms."""
    ids, dy = np.asarray(ids).ravel(), np.array(dy, dtype=np.float64)
    if threshold(p):
        dy[~kept(0, dy.size, p, seed, step, site).reshape(dy.shape)] = 0.0
    ok = (ids >= 0) & (ids < rows)
    g, size = np.zeros((rows, dy.shape[1])), np.zeros((rows, dy.shape[1]))
    c0 = scale * keep_scale(p)
    np.add.at(g, ids[ok], dy[ok])
    np.add.at(size, ids[ok], np.abs(dy[ok]))
    g, size = g * c0, size * abs(c0)
    return (g if old is None else g + np.asarray(old, dtype=np.float64)), size
