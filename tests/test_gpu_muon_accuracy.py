"""Spectra and ranks of the orthogonalised matrix on the GPU, in every form of the kernels.

Bounds (2-norm), u = 2^-8 the half step of bf16, r = oracle.muon.rounding_bound:
  * against the exact result: 2 r (what a call gives is about 0.7 r, and 1.8 r where a single value
    is rounded), and u |O| for the output;
  * against the oracle with the same roundings: of sums of K <= 500 terms in fp32 a part of at most
    K 2^-24 / 2^-11 < 1 / 12 lies so close to a tie that it is rounded the other way, by a step, whose mean
    square is 12 times a rounding's: r for the fp32 result, and 2 u |O| for outputs rounded
    apart.
"""
import numpy as np
import pytest
import torch

import gradient_sync_zero_amd as G
from oracle import muon as O
from tests import test_gpu_muon as updates
from tests.test_gpu_muon import f64, norm, run, workspace
from tests.test_muon_accuracy import STATED, U, far_eps, matrix, stated

pytestmark = pytest.mark.gpu


# one block (both orientations), panels, products in tiles of 64, in pairs, tall
@pytest.mark.parametrize("rows,cols", [(60, 100), (128, 128), (250, 120), (90, 400), (500, 100), (160, 200), (300, 257), (140, 1200), (1200, 140)])
@pytest.mark.parametrize("name", STATED)
def test_spectra(rows, cols, name):
    x = torch.from_numpy(matrix(rows, cols, name)).cuda()
    out = f64(run(x))
    exact, r = O.orthogonalize(f64(x)), O.rounding_bound(f64(x))
    assert norm(out - exact) <= 2 * r + U * norm(exact), (norm(out - exact) / norm(exact), r / norm(exact))
    limit = stated(rows, cols, name)
    assert limit is None or norm(out - exact) <= limit * norm(exact), norm(out - exact) / norm(exact)
    same = O.orthogonalize(f64(x), rounded=True)
    assert norm(out - same) <= r + 2 * U * norm(same), norm(out - same) / norm(same)


@pytest.mark.parametrize("rows,cols", [(60, 100), (90, 400), (160, 200), (1200, 140)])
@pytest.mark.parametrize("name", STATED)
def test_updates(rows, cols, name):
    """The weights of an update, whose direction is the gradient: O is not rounded to bf16."""
    u = matrix(rows, cols, name)
    plan = G.Plan([11, rows * cols], 1 << 40, 1)
    w, m, g = (torch.zeros(plan.flat_len, device="cuda") for _ in range(3))
    p = torch.zeros(plan.flat_len, dtype=torch.bfloat16, device="cuda")
    plan.view(1, g).copy_(torch.from_numpy(u).cuda().view(-1))
    hp = G.make_muon_hp(lr=1.0, momentum=0.0, scale=-1.0, nesterov=False)
    G.muon_step(plan, [1], rows, cols, w, m, g, torch.ones(1, device="cuda"), hp, p, workspace(1, rows, cols))
    got, exact = f64(plan.view(1, w)).reshape(rows, cols), O.orthogonalize(u)
    assert norm(got - exact) <= 2 * O.rounding_bound(u), norm(got - exact) / norm(exact)
    assert norm(got - O.orthogonalize(u, rounded=True)) <= O.rounding_bound(u)


# panels in both orientations, of one matrix and several; pairs of steps in both
@pytest.mark.parametrize("rows,cols,numel,tensors", [
    (300, 100, [5, 30000, 30000], [2, 1]), (100, 300, [30000, 3], [0]), (33, 2049, [67617, 9, 67617, 67617], [0, 3, 2]),
    (1000, 128, [128000], [0]), (140, 1200, [7, 168000, 168000], [1, 2]), (1200, 140, [168000, 1], [0])])
@pytest.mark.parametrize("nesterov", [True, False])
def test_update_with_a_long_side(rows, cols, numel, tensors, nesterov):
    """As tests/test_gpu_muon.py's updates: momentum bit for bit, weights, parameters, and what lies around."""
    updates.test_update(rows, cols, numel, tensors, nesterov)


def test_how_a_matrix_goes_depends_on_its_group():
    """Of 257 matrices of 129 x 400 the first 256 take steps in pairs and the last, alone, does not.  The
    update's O is fp32: nearer to the oracle with the same roundings (1e-3, tests/test_gpu_muon.py) than
    to the other one, and the last matrix has the bits it has by itself."""
    rows, cols, count = 129, 400, 257
    n = rows * cols
    plan = G.Plan([n] * count, 1 << 40, 1)
    g = torch.from_numpy(np.random.default_rng(1).normal(size=plan.flat_len).astype(np.float32)).cuda()
    hp = G.make_muon_hp(lr=1.0, momentum=0.0, scale=-1.0, nesterov=False)

    def update(tensors):
        w, m = torch.zeros_like(g), torch.zeros_like(g)
        p = torch.zeros(plan.flat_len, dtype=torch.bfloat16, device="cuda")
        G.muon_step(plan, tensors, rows, cols, w, m, g, torch.ones(1, device="cuda"), hp, p, workspace(len(tensors), rows, cols))
        return w

    w = update(range(count))
    assert torch.equal(plan.view(count - 1, update([count - 1])), plan.view(count - 1, w))
    for t in (0, 255, 256):
        u, got = f64(plan.view(t, g)).reshape(rows, cols), f64(plan.view(t, w)).reshape(rows, cols)
        as_paired, as_single = O.orthogonalize(u, rounded=True, count=256), O.orthogonalize(u, rounded=True)
        same, other = (as_single, as_paired) if t == 256 else (as_paired, as_single)
        assert np.array_equal(O.orthogonalize(u, rounded=True, count=count, index=t), same)
        assert norm(got - same) <= 1e-3 * norm(same)
        assert norm(got - same) < norm(got - other)


@pytest.mark.parametrize("eps", [1.0, 1e3, 1e6, 1e9, 1e12])
@pytest.mark.parametrize("rows,cols", [(40, 60), (90, 400), (140, 300)])
def test_eps_far_above_the_norm(rows, cols, eps):
    x = matrix(rows, cols, "random")
    x = torch.from_numpy(x / np.float32(norm(x))).cuda()
    exact, bound = far_eps(f64(x), eps)
    assert norm(f64(run(x, eps=eps)) - exact) <= bound
