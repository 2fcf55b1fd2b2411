"""Newton-Schulz orthogonalisation and the Muon update in 64 bits, and the same with the
library's roundings of the iterates to fp16."""
from __future__ import annotations

import numpy as np

NS = (3.4445, -4.7750, 2.0315)
SCALE_X, SCALE_A, SCALE_P = 2.0 ** 13, 2.0 ** 12, 2.0 ** 8   # the library holds 2^13 X, 2^12 A, 2^12 S and 2^8 S1 S0 in fp16


def _half(v, scale):
    return (v * scale).astype(np.float16).astype(np.float64) / scale


def in_pairs(rows, cols, count=1):
    """Whether the library takes two steps at once (X <- S1 S0 X, A1 = S0 A0 S0) for `count` matrices."""
    m, n = min(rows, cols), max(rows, cols)
    saved = count * m * m * (n - m)
    return m > 128 and (n >= 8 * m or (2 * n >= 5 * m and saved >= 1 << 30) or (2 * n >= 3 * m and saved >= 1 << 33))


def orthogonalize(x, steps=5, ns=None, eps=1e-7, rounded=False, count=1):
    """X = x / (|x| + eps); steps times A = X X^T, X = S X with S = a I + b A + c A A, from the
    smaller side.  rounded: X, A and S (and what a pair of steps adds) are rounded to fp16 where the
    library rounds them in a call of `count` such matrices."""
    x = np.asarray(x, dtype=np.float64)
    if x.shape[0] > x.shape[1]:
        return orthogonalize(x.T, steps, ns, eps, rounded, count).T
    x = x / (np.sqrt((x * x).sum()) + eps)
    half = _half if rounded else lambda v, scale: v
    pairs, k = rounded and in_pairs(*x.shape, count), 0

    def polynomial(A, k):
        a, b, c = NS if ns is None else ns[k]
        return half(a * np.eye(len(A)) + b * A + c * (A @ A), SCALE_A)

    while k < steps:
        if rounded:
            x = _half(x.astype(np.float32), SCALE_X)
        A = half(x @ x.T, SCALE_A)
        S = polynomial(A, k)
        if pairs and k + 2 <= steps and not (steps % 2 and k + 3 == steps and steps > 3):
            A = half(S @ half(S @ A, SCALE_A), SCALE_A)
            x = half(polynomial(A, k + 1) @ S, SCALE_P) @ x
            k += 2
        else:
            x = S @ x
            k += 1
    return x


def rounding_bound(x, steps=5, ns=None, eps=1e-7):
    """How far (2-norm) the fp16 roundings can take the result, to first order.

    f(s) = a s + b s^3 + c s^5 acts on the singular values.  A change E of X changes f(X) by at
    most L |E|, L the largest |f'| on [0, s_max] (the divided differences of f on [-s_max, s_max]
    are means of f').  Rounding is off by at most h = 2^-11 of a value: of X, |E| <= h |X|; of
    A = X X^T, S changes by b E + c (A E + E A), so X by (|b| + 2 |c| s^2) s h |A|; of S, by s h |S|."""
    x = np.asarray(x, dtype=np.float64)
    s = np.linalg.svd(x, compute_uv=False)
    s = s / (np.sqrt((s * s).sum()) + eps)
    h, bound = 2.0 ** -11, 0.0
    n2 = lambda v: float(np.sqrt((v * v).sum()))  # noqa: E731
    for k in range(steps):
        a, b, c = NS if ns is None else ns[k]
        top = float(s.max())
        t = np.linspace(0.0, top + bound, 2001)
        slope = float(np.abs(a + 3 * b * t ** 2 + 5 * c * t ** 4).max())
        bound = slope * (bound + h * n2(s))
        bound += (abs(b) + 2 * abs(c) * top ** 2) * top * h * n2(s * s) + top * h * n2(a + b * s ** 2 + c * s ** 4)
        s = np.abs(a * s + b * s ** 3 + c * s ** 5)
        if bound > 1.0:                              # past first order: nothing is promised
            return float("inf")
    return bound


def update(theta, m, g, coef, lr, mu, decay, scale, nesterov, rounded=False, **kw):
    """(theta, m, O) after the update, in 64 bits from the fp32 arrays."""
    gc = g.astype(np.float64) * float(coef)
    m = mu * m.astype(np.float64) + gc
    o = orthogonalize(gc + mu * m if nesterov else m, rounded=rounded, **kw)
    return theta.astype(np.float64) * (1.0 - lr * decay) - lr * scale * o, m, o
