"""The oracles of the orthogonalising update and the relative position bias against other
formulas: singular values, differences, and the published bucket values of the usual sizes."""
import numpy as np
import pytest

from oracle import muon, relpos


@pytest.mark.parametrize("r,c", [(1, 1), (5, 9), (12, 4), (30, 30)])
def test_newton_schulz_acts_on_the_singular_values(r, c):
    x = np.random.default_rng(r * 100 + c).normal(size=(r, c))
    u, s, v = np.linalg.svd(x, full_matrices=False)
    s = s / (np.linalg.norm(s) + 1e-7)
    for _ in range(5):
        s = 3.4445 * s - 4.7750 * s ** 3 + 2.0315 * s ** 5
    assert np.abs(muon.orthogonalize(x) - (u * s) @ v).max() < 1e-12


def test_other_coefficients_and_steps():
    x = np.random.default_rng(3).normal(size=(6, 10))
    # the cubic iteration converges to the polar factor
    u, _, v = np.linalg.svd(x, full_matrices=False)
    got = muon.orthogonalize(x, steps=40, ns=[(1.5, -0.5, 0.0)] * 40)
    assert np.abs(got - u @ v).max() < 1e-12


@pytest.mark.parametrize("r,c", [(16, 40), (60, 60), (90, 33)])
def test_the_roundings_stay_within_their_bound(r, c):
    x = np.random.default_rng(r).normal(size=(r, c))
    exact = muon.orthogonalize(x)
    off = np.linalg.norm(muon.orthogonalize(x, rounded=True) - exact)
    assert 0 < off < muon.rounding_bound(x)


def test_update_is_momentum_then_orthogonal():
    rng = np.random.default_rng(1)
    th, m, g = (rng.normal(size=(4, 7)).astype(np.float32) for _ in range(3))
    th1, m1, o = muon.update(th, m, g, 0.5, 0.1, 0.9, 0.2, 2.0, True)
    assert np.allclose(m1, 0.9 * m + 0.5 * g)
    assert np.allclose(o, muon.orthogonalize(0.5 * g + 0.9 * m1))
    assert np.allclose(th1, th * (1 - 0.02) - 0.2 * o)


def test_usual_borders():
    # 32 buckets in two directions up to 128, and in one
    assert relpos.borders(32, 128, True) == [0, 1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 23, 32, 46, 64, 91]
    one = relpos.borders(32, 128, False)
    assert one[:17] == list(range(17)) and one[17:] == [19, 21, 24, 27, 31, 35, 40, 46, 52, 59, 67, 77, 87, 99, 113]


@pytest.mark.parametrize("buckets,far,both", [(32, 128, True), (32, 128, False), (8, 20, True), (54, 333, True),
                                               (2, 2, False), (4, 2, True), (5, 3, False), (128, 4000, False)])
def test_borders_follow_the_logarithms(buckets, far, both):
    half = buckets // 2 if both else buckets
    e = half // 2
    d = np.arange(-2 * far, 2 * far)
    dist = np.abs(d) if both else np.maximum(-d, 0)
    want = e + np.floor(np.log(np.maximum(dist, 1) / e) / np.log(far / e) * (half - e) + 1e-9)
    want = np.where(dist < e, dist, np.minimum(half - 1, want)) + (half * (d > 0) if both else 0)
    assert np.array_equal(relpos.bucket(d, buckets, far, both), want)


def test_gradient_is_the_difference_of_the_bias():
    rng = np.random.default_rng(8)
    table, dy = rng.normal(size=(8, 3)), rng.normal(size=(2, 3, 9, 14))
    starts = [2, -5]
    g, _ = relpos.grad(dy, starts, 8, 20, True, 0.5)
    for b in range(8):
        for h in range(3):
            e = np.zeros_like(table)
            e[b, h] = 1.0
            diff = (dy * (relpos.bias(table + e, starts, 9, 14, 20, True, 0.5) - relpos.bias(table - e, starts, 9, 14, 20, True, 0.5))).sum() / 2
            assert abs(diff - g[b, h]) < 1e-12
