"""What oracle.muon.rounding_bound says against what the fp16 roundings do, and that a result with a
mistake in it is outside of the tolerances built on it (2 rounding_bound for fp32 results, half a
step of bf16 more for bf16 ones)."""
import numpy as np
import pytest

import gradient_sync_zero_amd as G
from oracle import muon

U = 2.0 ** -8


def norm(x):
    return float(np.sqrt((np.asarray(x) ** 2).sum()))


def spectrum(name, m):
    if name == "1e-3" or name == "1e-6":
        return 10.0 ** -np.linspace(0, float(name[3:]), m)
    return np.r_[np.ones(int(name)), np.zeros(m - int(name))]


def matrix(rows, cols, name, seed=1):
    """Random elements, singular values that fall evenly, or `name` equal ones and zeros."""
    rng = np.random.default_rng(seed)
    if name == "random":
        return rng.normal(size=(rows, cols)).astype(np.float32)
    m = min(rows, cols)
    u, v = np.linalg.qr(rng.normal(size=(rows, m)))[0], np.linalg.qr(rng.normal(size=(cols, m)))[0]
    return ((u * spectrum(name, m)) @ v.T).astype(np.float32)


NAMES = ["random", "1e-3", "1e-6", "1", "4", "8"]


@pytest.mark.parametrize("rows,cols", [(17, 64), (60, 100), (160, 200), (500, 200), (140, 1200)])
@pytest.mark.parametrize("name", NAMES)
def test_the_bound_is_near_what_the_roundings_do(rows, cols, name):
    """Each error is at most 1 and at least 1 / 2 of its part of the bound (the mean square of
    4^e / v^2, v in [2^e, 2^(e + 1)), is between 1 / 4 and 1), and pairs count one error twice."""
    x = matrix(rows, cols, name)
    off = norm(muon.orthogonalize(x, rounded=True) - muon.orthogonalize(x))
    assert 0.4 < off / muon.rounding_bound(x) < 1.0


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (5, 1), (2, 3), (4, 4), (1, 3001), (9, 5)])
def test_few_values(rows, cols):
    """A rounding alone is at most sqrt(3) of its mean square's root."""
    for seed in range(20):
        x = matrix(rows, cols, "random", seed)
        assert norm(muon.orthogonalize(x, rounded=True) - muon.orthogonalize(x)) <= 2 * muon.rounding_bound(x)


@pytest.mark.parametrize("steps,ns", [(1, None), (3, None), (16, None), (4, [(1.5, -0.5, 0.0)] * 3 + [(1.875, -1.25, 0.375)])])
@pytest.mark.parametrize("rows,cols", [(70, 150), (140, 1200)])
def test_other_steps(rows, cols, steps, ns):
    x = matrix(rows, cols, "random")
    off = norm(muon.orthogonalize(x, steps, ns, rounded=True) - muon.orthogonalize(x, steps, ns))
    bound = muon.rounding_bound(x, steps, ns)
    assert 0.1 * bound < off <= bound


def test_nothing_and_too_much():
    assert muon.rounding_bound(np.zeros((3, 4))) == 0.0
    with pytest.raises(ValueError, match="range"), np.errstate(all="ignore"):
        muon.rounding_bound(np.eye(3), 16, [(1e4, 1e4, 1e4)] * 16)


def bf16(v):
    w = np.ascontiguousarray(v, dtype=np.float32).view(np.uint32)
    return ((w + 0x7FFF + (w >> 16 & 1)) & np.uint32(0xFFFF0000)).view(np.float32).astype(np.float64)


@pytest.mark.parametrize("rows,cols", [(48, 96), (60, 100), (128, 128), (200, 500)])
def test_a_mistake_is_seen(rows, cols):
    x = matrix(rows, cols, "random")
    exact, good = muon.orthogonalize(x), muon.orthogonalize(x, rounded=True)
    update = 2 * muon.rounding_bound(x)
    out = update + U * norm(exact)
    assert norm(good - exact) <= update and norm(bf16(good) - exact) <= out
    a, b, c = muon.NS
    for wrong in (muon.orthogonalize(x, steps=4, rounded=True), muon.orthogonalize(x, ns=[(a, b, 1.02 * c)] * 5, rounded=True)):
        assert norm(bf16(wrong) - exact) > out
    part = bf16(good)
    part[-5:] = 0.0                                      # rows past the last whole tile left out
    assert norm(part - exact) > out
    part = bf16(good)
    part[0, 0] = np.nan
    assert not norm(part - exact) <= out
    assert norm(muon.orthogonalize(x, ns=[(a, b, 1.005 * c)] * 5) - exact) > update
    coarse = x.astype(np.float64) / norm(x)              # the iterates held in bf16
    for _ in range(5):
        coarse = bf16(coarse)
        A = bf16(coarse @ coarse.T)
        coarse = bf16(a * np.eye(rows) + b * A + c * A @ A) @ coarse
    assert norm(coarse - exact) > update


@pytest.mark.parametrize("name", ["1e-3", "1e-6", "1", "8"])
def test_a_mistake_is_seen_in_other_spectra(name):
    x = matrix(60, 100, name)
    exact, a = muon.orthogonalize(x), muon.NS[0]
    out = 2 * muon.rounding_bound(x) + U * norm(exact)
    assert norm(bf16(muon.orthogonalize(x, rounded=True)) - exact) <= out
    for wrong in (muon.orthogonalize(x, steps=4), muon.orthogonalize(x, ns=[(0.9 * a, *muon.NS[1:])] * 5)):
        assert norm(bf16(wrong) - exact) > out


def test_groups():
    """How many matrices go together, and so whether in pairs, as the library's host half has it: a
    workspace grows with the group alone, and holds the pairs' matrix where there are any."""
    assert [muon.group_of(129, 400, 257, k) for k in (0, 255, 256)] == [256, 256, 1]
    assert [muon.group_of(2 ** 17, 2 ** 14, 9, k) for k in (0, 3, 4, 8)] == [4, 4, 4, 1]
    assert muon.group_of(65536, 65536, 5) == 2 and muon.group_of(3, 2, 1) == 1
    assert muon.in_pairs(129, 400, 256) and not muon.in_pairs(129, 400, 1)
    size = lambda *a: G.muon_workspace_bytes(*a)  # noqa: E731
    assert size(255, 129, 400) < size(256, 129, 400) == size(257, 129, 400) == size(10 ** 6, 129, 400)
    assert size(3, 2 ** 17, 2 ** 14) < size(4, 2 ** 17, 2 ** 14) == size(9, 2 ** 17, 2 ** 14)


def test_a_matrix_behind_the_first_groups():
    x = matrix(129, 400, "random")
    first, last, alone = (muon.orthogonalize(x, rounded=True, **kw) for kw in (dict(count=257), dict(count=257, index=256), {}))
    assert np.array_equal(last, alone) and not np.array_equal(first, last)


# What include/gsz.h states of five steps: parts of the exact result, its rounding to bf16 included.
STATED = {"random": (0.0025, 0.004), "1e-3": (0.01, 0.02), "1e-6": (0.02, 0.03), "32": (0.03, None), "16": (0.05, 0.04), "8": (0.045, 0.045),
          "4": (0.085, 0.085), "1": (0.16, 0.16)}


def stated(rows, cols, name):
    """The limit for a matrix of these sizes, or None where none is stated."""
    m = min(rows, cols)
    if m < 16:
        return 0.006 if name == "random" else 0.16
    limit = STATED[name][m < 64]
    return None if name == "16" and m < 32 else limit


@pytest.mark.parametrize("rows,cols", [(1, 40), (2, 3), (4, 4), (12, 30), (17, 64), (60, 60), (33, 2049), (60, 100), (64, 64), (128, 128), (160, 200),
                                       (140, 1200), (500, 200), (300, 2400), (512, 512)])
def test_the_stated_accuracy(rows, cols):
    for name in STATED:
        if name != "random" and (min(rows, cols) < 3 or name.isdigit() and int(name) >= min(rows, cols)) or stated(rows, cols, name) is None:
            continue
        for seed in range(3):
            x = matrix(rows, cols, name, seed)
            exact = muon.orthogonalize(x)
            off = norm(bf16(muon.orthogonalize(x, rounded=True)) - exact) / norm(exact)
            assert off <= stated(rows, cols, name), (name, seed, off)


def test_positive_rank_one():
    rng = np.random.default_rng(3)
    for rows, cols in ((128, 128), (140, 1200), (300, 2400)):
        x = np.outer(rng.uniform(0.1, 1, rows), rng.uniform(0.1, 1, cols)).astype(np.float32)
        exact = muon.orthogonalize(x)
        assert norm(bf16(muon.orthogonalize(x, rounded=True)) - exact) <= 0.16 * norm(exact)


def far_eps(x, eps):
    """How far the result may be off where eps is far above |x|, and fp16 has no full precision: each
    of the 5 roundings of X is off by 2^-38 an element, grown by a = 3.4445 a step; X elsewhere and S by 2^-11
    of their values, and the output by its own rounding."""
    exact = muon.orthogonalize(x, eps=eps)
    absolute = 2.0 ** -38 * sum(muon.NS[0] ** k for k in range(1, 6))
    assert absolute < 3e-9
    return exact, absolute * np.sqrt(x.size) + (10 * 2.0 ** -11 + U) * norm(exact)


@pytest.mark.parametrize("eps", [1.0, 1e3, 1e6, 1e9, 1e12])
@pytest.mark.parametrize("rows,cols", [(40, 60), (140, 300)])
def test_eps_far_above_the_norm(rows, cols, eps):
    x = matrix(rows, cols, "random")
    x = (x / norm(x)).astype(np.float32)
    exact, bound = far_eps(x, eps)
    assert norm(bf16(muon.orthogonalize(x, eps=eps, rounded=True)) - exact) <= bound
