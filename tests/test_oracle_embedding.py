"""The 64-bit embedding and dropout oracle pinned to what it must be: Philox's
published known answers, the mask's rate and its exact expectation, and the
gradient as the derivative of the lookup (by differences, which are exact up to
rounding: the lookup is linear in the table)."""
import os

import numpy as np
import pytest

from oracle import embedding as E


def test_philox_known_answers():
    path = os.path.join(os.path.dirname(__file__), "golden", "philox4x32_10_kat.txt")
    n = 0
    for line in open(path):
        f = line.split("#")[0].split()
        if not f:
            continue
        v = [int(x, 16) for x in f[-10:]]
        got = E.philox4x32_10([np.array([x]) for x in v[:4]], v[4:6])
        assert [int(x[0]) for x in got] == v[6:], line
        n += 1
    assert n >= 3


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.97, 2.0 ** -20, 1.0 - 2.0 ** -40])
def test_mask_rate_is_p(p):
    n = 1 << 18
    dropped = n - int(E.kept(0, n, p, 12345678901234567, 3, 9).sum())
    q = E.threshold(p) / 2.0 ** 32
    # six standard deviations of a binomial count (and all or nothing at the ends)
    assert abs(dropped - n * q) <= 6 * np.sqrt(n * q * (1 - q)) + 1e-9 * n
    assert E.keep_scale(p) * (1 - q) == pytest.approx(1.0, rel=1e-15)
    assert q <= p and p - q < 2.0 ** -32


def test_mask_depends_on_element_seed_step_and_site_alone():
    base = E.numbers(0, 4096, 77, 5, 2)
    assert np.array_equal(base[100:1003], E.numbers(100, 903, 77, 5, 2))
    assert np.array_equal(base, E.numbers(0, 4096, 77, 5 + (1 << 32), 2))     # the step is taken mod 2^32
    for other in ((78, 5, 2), (77 + (1 << 32), 5, 2), (77, 6, 2), (77, 5, 3)):
        assert (base != E.numbers(0, 4096, *other)).mean() > 0.99
    # halves are 16-bit numbers of their own: no two of the eight are alike over the blocks
    cols = base.reshape(-1, 8)
    assert all((cols[:, i] != cols[:, j]).mean() > 0.99 for i in range(8) for j in range(i))


def test_grad_is_the_derivative_of_the_lookup():
    rng = np.random.default_rng(4)
    rows, dim, n = 11, 5, 40
    ids = rng.integers(-2, rows + 2, n)
    table, dy = rng.normal(size=(rows, dim)), rng.normal(size=(n, dim))
    kw = dict(scale=1.7, p=0.3, seed=99, step=4, site=1)
    g, _ = E.grad(ids, dy, rows, **kw)
    base = (E.lookup(ids, table, **kw) * dy).sum()
    for v in range(rows):
        for c in range(dim):
            t = table.copy()
            t[v, c] += 1.0
            assert (E.lookup(ids, t, **kw) * dy).sum() - base == pytest.approx(g[v, c], abs=1e-11)
    old = rng.normal(size=(rows, dim))
    assert np.allclose(E.grad(ids, dy, rows, old=old, **kw)[0], old + g, rtol=0, atol=1e-15)


def test_dropout_backward_is_dropout():
    rng = np.random.default_rng(5)
    x, dy = rng.normal(size=333), rng.normal(size=333)
    a = (5, 6, 7)
    # <dropout(x), dy> = <x, dropout(dy)>: the map is its own transpose
    assert (E.dropout(x, 0.4, *a) * dy).sum() == pytest.approx((x * E.dropout(dy, 0.4, *a)).sum(), rel=1e-14)
