"""Newton-Schulz orthogonalisation and the Muon update in 64 bits, and the same with the
library's roundings of the iterates to fp16."""
from __future__ import annotations

import numpy as np

NS = (3.4445, -4.7750, 2.0315)
SCALE_X, SCALE_A, SCALE_P = 2.0 ** 13, 2.0 ** 12, 2.0 ** 8   # the library holds 2^13 X, 2^12 A, 2^12 S and 2^8 S1 S0 in fp16


def _half(v, scale):
    return (v * scale).astype(np.float16).astype(np.float64) / scale


def group_of(rows, cols, count, index=0):
    """How many matrices matrix `index` of a call's `count` goes with: 256 at a time, fewer where they
    would have more than 2^33 elements (sides rounded up to 64), the rest at the end."""
    padded = -(-rows // 64) * 64 * (-(-cols // 64) * 64)
    most = max(1, min(256, 2 ** 33 // padded))
    return min(most, count - index // most * most)


def in_pairs(rows, cols, count=1):
    """Whether the library takes two steps at once (X <- S1 S0 X, A1 = S0 A0 S0) for a group of `count`
    matrices."""
    m, n = min(rows, cols), max(rows, cols)
    saved = count * m * m * (n - m)
    return m > 128 and (n >= 8 * m or (2 * n >= 5 * m and saved >= 1 << 30) or (2 * n >= 3 * m and saved >= 1 << 33))


def launches(steps, pairs):
    """(first step, how many) of what goes at once: in pairs, of an odd number the one before the last
    pair alone."""
    k = 0
    while k < steps:
        many = 2 if pairs and k + 2 <= steps and not (steps % 2 and k + 3 == steps and steps > 3) else 1
        yield k, many
        k += many


def orthogonalize(x, steps=5, ns=None, eps=1e-7, rounded=False, count=1, index=0):
    """X = x / (|x| + eps); steps times A = X X^T, X = S X with S = a I + b A + c A A, from the
    smaller side.  rounded: X, A and S (and what a pair of steps adds) are rounded to fp16 where the
    library rounds them in matrix `index` of a call of `count`."""
    x = np.asarray(x, dtype=np.float64)
    if x.shape[0] > x.shape[1]:
        return orthogonalize(x.T, steps, ns, eps, rounded, count, index).T
    x = x / (np.sqrt((x * x).sum()) + eps)
    half = _half if rounded else lambda v, scale: v

    def polynomial(A, k):
        a, b, c = NS if ns is None else ns[k]
        return half(a * np.eye(len(A)) + b * A + c * (A @ A), SCALE_A)

    for k, many in launches(steps, rounded and in_pairs(*x.shape, group_of(*x.shape, count, index))):
        if rounded:
            x = _half(x.astype(np.float32), SCALE_X)
        A = half(x @ x.T, SCALE_A)
        S = polynomial(A, k)
        if many == 2:
            A = half(S @ half(S @ A, SCALE_A), SCALE_A)
            S = half(polynomial(A, k + 1) @ S, SCALE_P)
        x = S @ x
    return x


def rounding_bound(x, steps=5, ns=None, eps=1e-7, count=1, index=0):
    """How far (2-norm) the fp16 roundings take the result: the root of the mean square over roundings,
    to first order.  What a call gives is 0.6 to 0.75 of it where many values are rounded (they lie anywhere
    between powers of two) and can be 1.8 times it where there is one.

    A rounding to fp16 is off by up to half a step of 2^-10 of the power of two below the value,
    evenly: in the mean square by r = 2^-10 / sqrt(12) of the value at most.  An error of X keeps its mean
    square in the singular vectors' basis, where f(s) = a s + b s^3 + c s^5 takes its symmetric part
    in (i, j) times (f(si) - f(sj)) / (si - sj), its antisymmetric part times (f(si) + f(sj)) / (si + sj) and what
    lies outside of the smaller side times f(si) / si.  An error E of A is one of (b + c (li + lj)) E of
    S, l = s^2, and an error D of S one of D sj of the next X.  Of a pair of steps A1 = S0 (S0 A0) and S1 S0 are
    written from their lower halves: where a factor's error makes a product unsymmetric, half of it is
    the other side's."""
    x = np.asarray(x, dtype=np.float64)
    m, n = sorted(x.shape)
    s = np.linalg.svd(x, compute_uv=False)
    s = s / (np.sqrt((s * s).sum()) + eps)
    if not s.any():
        return 0.0
    r2 = 2.0 ** -20 / 12
    col, row = (lambda v: v[:, None]), (lambda v: v[None])

    def quotient(x, y, a, b, c):                     # (f(x) - f(y)) / (x - y)
        return a + b * (x * x + x * y + y * y) + c * (x ** 4 + x ** 3 * y + x * x * y * y + x * y ** 3 + y ** 4)

    def rounding(values):                            # of an element of a matrix with these eigenvalues
        return r2 * (values ** 2).sum() / m ** 2

    same, anti, outside = np.zeros((m, m)), np.zeros((m, m)), np.zeros(m)    # mean squares of X's error
    for k, many in launches(steps, in_pairs(m, n, group_of(m, n, count, index))):
        e = r2 * (s * s).sum() / (m * n)
        same, anti, outside = same + e / 2, anti + e / 2, outside + (n - m) * e
        s0, ea = s, rounding(s * s)
        for j in range(many):
            a, b, c = NS if ns is None else ns[k + j]
            l = s * s                                # noqa: E741
            p = a + b * l + c * l * l
            es = (b + c * (col(l) + row(l))) ** 2 * ea + rounding(p)
            same = same * quotient(col(s), row(s), a, b, c) ** 2 + es * (col(s) + row(s)) ** 2 / 4
            anti = anti * quotient(col(s), -row(s), a, b, c) ** 2 + es * (col(s) - row(s)) ** 2 / 4
            outside = outside * p ** 2
            if many == 2 and j == 0:
                et = rounding(p * l) + es * (col(l) - row(l)) ** 2 / 2
                ea = (col(p) * row(p)) ** 2 * ea + (col(p) ** 2 + (col(p) - row(p)) ** 2 / 2) * et + rounding((p * s) ** 2)
                p0, es0 = p, es
            elif many == 2:
                es = rounding(p * p0) + (es * (col(p0) - row(p0)) ** 2 + es0 * (col(p) - row(p)) ** 2) / 2
                same, anti = same + es * (col(s0) + row(s0)) ** 2 / 4, anti + es * (col(s0) - row(s0)) ** 2 / 4
            s = s * p
    total = float(np.sqrt(same.sum() + anti.sum() + outside.sum()))
    if not np.isfinite(total):
        raise ValueError("the iteration leaves the range of the first order")
    return total


def update(theta, m, g, coef, lr, mu, decay, scale, nesterov, rounded=False, **kw):
    """(theta, m, O) after the update, in 64 bits from the fp32 arrays."""
    gc = g.astype(np.float64) * float(coef)
    m = mu * m.astype(np.float64) + gc
    o = orthogonalize(gc + mu * m if nesterov else m, rounded=rounded, **kw)
    return theta.astype(np.float64) * (1.0 - lr * decay) - lr * scale * o, m, o
