"""The orthogonalising kernels run on the CPU (tests/muon_values_host.cpp) value by value against
the 64-bit oracle, so that a NaN anywhere fails: the workspace holds NaNs before the call."""
import subprocess

import numpy as np
import pytest

from oracle import muon as O
from oracle.plan import make_plan
from tests.test_muon_accuracy import U, matrix, norm
from tests.test_optim_host import build


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    return build(tmp_path_factory, "muon_values_host", "tests/host_matrix", "tests/host_gpu", "include", "gradient_sync_zero_amd/optim",
                 "gradient_sync_zero_amd/csrc")


def run(exe, tmp_path, values, *args):
    values.tofile(tmp_path / "in")
    r = subprocess.run([exe, *map(str, args), tmp_path / "in", tmp_path / "out"], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, (r.returncode, r.stderr[-2000:])
    return np.fromfile(tmp_path / "out", dtype=np.uint16)


def widen(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def nearest(v):
    w = v.astype(np.float32).view(np.uint32)
    return ((w + 0x7FFF + (w >> 16 & 1)) >> 16).astype(np.uint16)


# one block, panels (both orientations), products, pairs of steps
@pytest.mark.parametrize("count,rows,cols,bf,steps", [
    (1, 1, 1, 0, 5), (2, 5, 9, 1, 5), (2, 96, 40, 0, 3), (1, 100, 256, 1, 2), (1, 33, 300, 1, 5), (2, 700, 100, 0, 2), (1, 1, 3000, 1, 5),
    (1, 129, 200, 0, 2), (1, 200, 129, 1, 2), (1, 130, 1100, 0, 3)])
def test_orthogonalize(host, tmp_path, count, rows, cols, bf, steps):
    x = np.stack([matrix(rows, cols, "random", seed) for seed in range(count)])
    if bf:
        x = widen(nearest(x.ravel())).reshape(x.shape)
    out = widen(run(host, tmp_path, nearest(x.ravel()) if bf else x, "orthogonalize", count, rows, cols, 0 if bf else 1, steps)).reshape(x.shape)
    for got, xi in zip(out, x):
        exact = O.orthogonalize(xi, steps)
        assert norm(got - exact) <= 2 * O.rounding_bound(xi, steps) + U * norm(exact)


@pytest.mark.parametrize("count,rows,cols,nesterov", [(1, 7, 5, 1), (3, 20, 33, 0), (1, 140, 30, 1), (2, 300, 100, 1), (2, 60, 300, 0), (1, 130, 200, 1)])
def test_update(host, tmp_path, count, rows, cols, nesterov):
    n = rows * cols
    plan = make_plan([k for b in range(count) for k in (n, 3 + b)], 1000, 2, 8)
    length = plan.flat_len
    rng = np.random.default_rng(count + rows)
    w0, m0, g = (rng.normal(0, std, length).astype(np.float32) for std in (0.02, 1.0, 0.3))
    bits = run(host, tmp_path, np.concatenate([w0, m0, g]), "step", count, rows, cols, nesterov)
    w1, m1 = bits[:4 * length].view(np.float32).reshape(2, length)
    p1 = bits[4 * length:]
    scale = 0.2 * max(rows, cols) ** 0.5
    other = np.ones(length, dtype=bool)
    for b in range(count):
        s = slice(plan.tensor_offset[2 * b], plan.tensor_offset[2 * b] + n)
        other[s] = False
        shape = lambda v: v[s].reshape(rows, cols)  # noqa: E731
        theta, m, o = O.update(shape(w0), shape(m0), shape(g), 0.75, 0.02, 0.95, 0.1, scale, bool(nesterov))
        # momentum: three roundings of half a step 2^-24, of values up to the terms' sizes
        assert (np.abs(shape(m1) - m) <= 3 * 2.0 ** -24 * (np.abs(0.95 * shape(m0)) + np.abs(0.75 * shape(g)))).all()
        u = 0.75 * shape(g).astype(np.float64) + 0.95 * m if nesterov else m
        # theta: the decay's, the product's and the sum's roundings
        assert norm(shape(w1) - theta) <= 0.02 * scale * 2 * O.rounding_bound(u) + 4 * 2.0 ** -24 * norm(theta)
        assert np.array_equal(p1[s], nearest(w1[s]))
    assert np.array_equal(w1[other], w0[other]) and np.array_equal(m1[other], m0[other]) and (p1[other] == 0x1234).all()
