"""Calls of the orthogonalising update that the form of the kernels matters to, in each form: one
block, panels, products in tiles, and pairs of steps.  What one form does is compared with the same
call in ordinary circumstances, bit for bit."""
import numpy as np
import pytest
import torch

import gradient_sync_zero_amd as G
from tests.test_gpu_muon import BF, F32, f64, run, run_keep, workspace

pytestmark = pytest.mark.gpu

# one block; panels; products of tiles of 64; tall; pairs of steps, both ways
FORMS = [(40, 60), (70, 1500), (900, 100), (260, 300), (500, 200), (140, 1200), (1200, 140)]


def matrices(count, rows, cols, dtype=F32):
    rng = np.random.default_rng(rows + cols)
    return torch.from_numpy(rng.normal(size=(count, rows, cols))).to(dtype).cuda()


@pytest.mark.parametrize("rows,cols", FORMS)
def test_zeros_and_values_that_are_not_finite_stay_in_their_matrix(rows, cols):
    x = matrices(5, rows, cols)
    want = run(x)
    x[1] = 0.0
    x[3, rows - 1, cols - 1] = float("inf")
    x[4, 0, 0] = float("nan")
    out = run_keep(x)
    assert bool((out[1] == 0).all()) and bool(out[3:].isnan().all())
    assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2])


@pytest.mark.parametrize("rows,cols", FORMS)
def test_in_place_and_unaligned(rows, cols):
    x = matrices(2, rows, cols, BF)
    want = run(x)
    for shift in (0, 1, 3):
        y = torch.empty(x.numel() + 8, dtype=BF, device="cuda")[shift:shift + x.numel()].view(x.shape)
        y.copy_(x)
        G.orthogonalize(y, y, workspace(2, rows, cols))
        assert torch.equal(y, want)
        z = torch.empty(x.numel() + 8, dtype=F32, device="cuda")[shift:shift + x.numel()].view(x.shape)
        z.copy_(x)
        G.orthogonalize(z, y.zero_(), workspace(2, rows, cols))
        assert torch.equal(y, want)


@pytest.mark.parametrize("rows,cols", FORMS)
def test_largest_and_smallest_numbers(rows, cols):
    """Powers of two scale every value and the norm alike: the same bits."""
    x = matrices(1, rows, cols)[0]
    want = run(x, eps=1e-30)
    for e in (-70, 100):
        assert torch.equal(run(x * 2.0 ** e, eps=1e-30), want)
    assert bool((run(torch.zeros_like(x), eps=1e-30) == 0).all())


@pytest.mark.parametrize("rows,cols", FORMS)
def test_captured_and_on_two_streams_at_once(rows, cols):
    plan = G.Plan([rows * cols, 7, rows * cols, rows * cols], 1 << 40, 1)
    rng = np.random.default_rng(rows)
    start = [torch.from_numpy(rng.normal(0, s, plan.flat_len).astype(np.float32)).cuda() for s in (0.02, 4e-3, 1e-3)]
    coef, hp = torch.tensor([0.5], device="cuda"), G.make_muon_hp(lr=0.02, scale=2.0, weight_decay=0.1)

    class State:
        def __init__(self):
            self.w, self.m, self.g = (t.clone() for t in start)
            self.p = torch.zeros(plan.flat_len, dtype=BF, device="cuda")
            self.ws = workspace(3, rows, cols)

        def step(self, stream=None):
            G.muon_step(plan, [3, 0, 2], rows, cols, self.w, self.m, self.g, coef, hp, self.p, self.ws, stream=stream)

        def same(self, other):
            return all(torch.equal(a, b) for a, b in ((self.w, other.w), (self.m, other.m), (self.p, other.p)))

    eager, captured = State(), [State(), State()]
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    torch.cuda.synchronize()
    for graph, state, stream in zip(graphs, captured, side):
        with torch.cuda.graph(graph, stream=stream):
            state.step()
    torch.cuda.synchronize()
    for k in range(3):
        for graph, stream in zip(graphs, side):             # two graphs with a workspace each, at once
            with torch.cuda.stream(stream):
                graph.replay()
        eager.step()
        torch.cuda.synchronize()
        for state in captured:
            assert state.same(eager), k
            state.ws.fill_(0xFF)
        torch.cuda.synchronize()
    for _ in range(3):
        for state, stream in zip(captured, side):
            state.step(stream)
        eager.step()
    torch.cuda.synchronize()
    assert all(state.same(eager) for state in captured)


@pytest.mark.parametrize("rows,cols", FORMS)
def test_clipped_to_nothing(rows, cols):
    """A coefficient of 0 and a momentum of 0: nothing to orthogonalise, the decay alone; one that is not
    finite reaches the listed matrices and no other."""
    plan = G.Plan([rows * cols, 9], 1 << 40, 1)
    g = torch.randn(plan.flat_len, device="cuda")
    w = torch.randn(plan.flat_len, device="cuda")
    keep, m = w.clone(), torch.zeros_like(w)
    p = torch.zeros(plan.flat_len, dtype=BF, device="cuda")
    hp = G.make_muon_hp(lr=0.25, scale=2.0, weight_decay=0.5)
    ws = workspace(1, rows, cols)
    G.muon_step(plan, [0], rows, cols, w, m, g, torch.zeros(1, device="cuda"), hp, p, ws)
    assert torch.equal(plan.view(0, w), plan.view(0, keep) * 0.875) and bool((m == 0).all())
    assert torch.equal(plan.view(1, w), plan.view(1, keep))
    G.muon_step(plan, [0], rows, cols, w, m, g, torch.full((1,), float("nan"), device="cuda"), hp, p, ws)
    assert bool(plan.view(0, w).isnan().all()) and bool(plan.view(0, p).isnan().all()) and bool(plan.view(0, m).isnan().all())
    assert torch.equal(plan.view(1, w), plan.view(1, keep)) and bool((f64(plan.view(1, p)) == 0).all())
