"""The relative position bias and its gradient on the GPU against the 64-bit oracle.

Bounds, with e = 2^-24 and u the half step of the output's type (bf16 2^-8, fp32 e):
  * bias: scale is rounded once, the product once, the sum once, the output once;
  * gradient: a bucket's partial sums add at most m = 256 + 32 + 8 values one after the other in fp32
    (a diagonal's in a tile, a lane's share of the diagonals, the wave), so they are off by m e of the
    terms' sizes at most; the join is fp64; one rounding.
"""
import numpy as np
import pytest
import torch

import gradient_sync_zero_amd as G
from oracle import relpos as O
from tests.test_gpu_embedding import BF, EPS, F32, U, Guarded, f64, near, out_bound

pytestmark = pytest.mark.gpu

# batch, heads, q, k, buckets, max_distance, both
SHAPES = [(1, 1, 1, 1, 2, 2, False), (2, 3, 17, 33, 8, 20, True), (3, 2, 1, 131, 32, 128, False), (1, 2, 70, 90, 10, 7, True),
          (1, 1, 300, 9, 32, 128, True), (1, 2, 40, 2100, 54, 333, False), (2, 1, 65, 64, 256, 300, True), (16, 12, 1, 1031, 32, 128, False),
          (1, 1, 1500, 1, 32, 128, True), (1, 3, 513, 515, 32, 128, False), (2, 2, 257, 4099, 64, 1000, True), (5, 7, 8, 8, 32, 128, True)]


def starts_for(kind, batch, q, k, rng):
    """(the argument, one number a sequence)"""
    if kind == "zero":
        return 0, [0] * batch
    if kind == "end":
        return k - q, [k - q] * batch
    v = rng.integers(-q, k + q, batch)
    return torch.from_numpy(v).to(torch.int32 if kind == "i32" else torch.int64).cuda(), v.tolist()


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("table,dtype,add,start,shift", [
    (BF, BF, True, "zero", 0), (F32, F32, False, "end", 1), (BF, F32, True, "i64", 3), (F32, BF, False, "i32", 5)])
def test_bias(shape, table, dtype, add, start, shift):
    batch, heads, q, k, buckets, far, both = shape
    rng = np.random.default_rng(q + k)
    t = Guarded((buckets, heads), table, shift, torch.from_numpy(rng.normal(size=(buckets, heads))).to(table).cuda())
    a = Guarded((batch, heads, q, k), dtype, 2 * shift, torch.from_numpy(rng.normal(size=(batch, heads, q, k))).to(dtype).cuda())
    out = Guarded((batch, heads, q, k), dtype, shift)
    arg, each = starts_for(start, batch, q, k, rng)
    scale = 0.7
    G.relpos_bias(t.t, out.t, far, both, q_start=arg, scale=scale, add=a.t if add else None)
    for x in (t, a, out):
        x.check()
    product = O.bias(f64(t.t), each, q, k, far, both, scale)
    ref = product + f64(a.t) if add else product
    bound = np.abs(product) * ((1 + EPS) ** 2 - 1) * (1 + U[dtype]) * (1 + EPS) + out_bound(ref, dtype, 1)
    near(out.t, ref, bound, "bias")
    if add:                                             # in place
        want = out.t.clone()
        G.relpos_bias(t.t, a.t, far, both, q_start=arg, scale=scale, add=a.t)
        assert torch.equal(a.t, want)


def test_masked_scores_stay_masked():
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.normal(size=(2, 2, 9, 20))).to(BF).cuda()
    x[0, :, 3] = -float("inf")                          # a row that leaves nothing
    x[1, 0, :, 7] = torch.finfo(BF).min
    x[1, 1, 2, 2] = float("nan")
    t = torch.from_numpy(rng.normal(size=(8, 2))).to(BF).cuda()
    out = torch.empty_like(x)
    G.relpos_bias(t, out, 20, add=x)
    assert bool((out[0, :, 3] == -float("inf")).all()) and bool((out[1, 0, :, 7] <= -3e38).all()) and bool(out[1, 1, 2, 2].isnan())
    assert int(out.isnan().sum()) == 1 and int(out.isinf().sum()) == 2 * 20


def test_single_tokens_are_rows_of_the_whole():
    """The bias of each new token of a sequence is the row that the whole prompt has for it."""
    heads, n = 3, 77
    t = torch.from_numpy(np.random.default_rng(2).normal(size=(32, heads))).to(F32).cuda()
    whole = torch.empty(1, heads, n, n, device="cuda")
    G.relpos_bias(t, whole, 128, False)
    place = torch.arange(n, device="cuda")
    rows = torch.empty(n, heads, 1, n, device="cuda")
    G.relpos_bias(t, rows, 128, False, q_start=place)
    assert torch.equal(rows[:, :, 0].transpose(0, 1), whole[0])


def test_far_starts():
    t = torch.arange(16, dtype=F32, device="cuda").view(8, 2)
    out = torch.empty(3, 2, 2, 5, device="cuda")
    big = 2 ** 62
    G.relpos_bias(t, out, 20, True, q_start=torch.tensor([-big, big, 0], device="cuda"))
    assert bool((out[0, 0] == t[7, 0]).all()) and bool((out[1, 1] == t[3, 1]).all())
    G.relpos_bias(t, out, 20, True, q_start=2 ** 40)
    assert bool((out[:, 0] == t[3, 0]).all())


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype,grad,acc,start,shift", [
    (BF, F32, True, "zero", 0), (F32, BF, False, "end", 1), (BF, BF, True, "i64", 3), (F32, F32, False, "i32", 5)])
def test_gradient(shape, dtype, grad, acc, start, shift):
    batch, heads, q, k, buckets, far, both = shape
    rng = np.random.default_rng(q * 3 + k)
    dy = Guarded((batch, heads, q, k), dtype, shift, torch.from_numpy(rng.normal(0, 1e-3, (batch, heads, q, k))).to(dtype).cuda())
    g = Guarded((buckets, heads), grad, 2 * shift, torch.from_numpy(rng.normal(0, 1e-2, (buckets, heads))).to(grad).cuda())
    old = f64(g.t).copy()
    arg, each = starts_for(start, batch, q, k, rng)
    nbytes = G.relpos_bias_workspace_bytes(batch, heads, q, k, buckets)
    ws = torch.full((nbytes + 16,), 0xFF, dtype=torch.uint8, device="cuda")
    G.relpos_bias_grad(dy.t, g.t, ws[:nbytes], far, both, q_start=arg, scale=0.7, accumulate=acc)
    dy.check()
    g.check()
    assert bool((ws[nbytes:] == 0xFF).all()), "wrote behind the workspace"
    ref, size = O.grad(f64(dy.t), each, buckets, far, both, 0.7, old if acc else None)
    near(g.t, ref, size * 296 * EPS * (1 + U[grad]) + out_bound(ref, grad, 1), "gradient")
    again = Guarded((buckets, heads), grad, 0, torch.from_numpy(old).to(grad).cuda())
    G.relpos_bias_grad(dy.t, again.t, ws[:nbytes], far, both, q_start=arg, scale=0.7, accumulate=acc)
    assert torch.equal(again.t, g.t), "the same call, other bits"


def test_gradient_is_the_transpose_of_the_bias():
    """<dy, bias(table)> = <grad(dy), table>, by differences in one bucket at a time."""
    rng = np.random.default_rng(9)
    heads, q, k, buckets = 2, 33, 47, 8
    dy = torch.from_numpy(rng.normal(size=(2, heads, q, k))).to(F32).cuda()
    g = torch.empty(buckets, heads, device="cuda")
    ws = torch.empty(G.relpos_bias_workspace_bytes(2, heads, q, k, buckets), dtype=torch.uint8, device="cuda")
    G.relpos_bias_grad(dy, g, ws, 20, True, q_start=5)
    out = torch.empty_like(dy)
    for b in range(buckets):
        t = torch.zeros(buckets, heads, device="cuda")
        t[b] = 1.0
        G.relpos_bias(t, out, 20, True, q_start=5)
        want = (f64(dy) * f64(out)).sum((0, 2, 3))
        assert np.abs(f64(g)[b] - want).max() <= 296 * EPS * np.abs(f64(dy)).sum()


def test_gradient_of_nothing_and_of_infinities():
    g = torch.full((8, 2), 3.0, device="cuda")
    for shape in ((0, 2, 3, 4), (1, 2, 0, 4), (1, 2, 3, 0)):
        G.relpos_bias_grad(torch.empty(shape, device="cuda"), g, None, 20, accumulate=True)
        assert bool((g == 3.0).all())
    G.relpos_bias_grad(torch.empty(1, 2, 3, 0, device="cuda"), g, None, 20)
    assert bool((g == 0.0).all())
    dy = torch.zeros(1, 2, 20, 20, device="cuda")
    dy[0, 1, 5, 5] = float("inf")
    dy[0, 0, 5, 6] = float("nan")
    ws = torch.empty(G.relpos_bias_workspace_bytes(1, 2, 20, 20, 8), dtype=torch.uint8, device="cuda")
    G.relpos_bias_grad(dy, g, ws, 20)
    assert float(g[0, 1]) == float("inf") and bool(g[5, 0].isnan()) and int((g == 0).sum()) == 14


def test_capture_and_other_streams():
    rng = np.random.default_rng(3)
    t = torch.from_numpy(rng.normal(size=(32, 4))).to(BF).cuda()
    x = torch.from_numpy(rng.normal(size=(2, 4, 100, 90))).to(BF).cuda()
    start = torch.tensor([3, 9], device="cuda")
    nbytes = G.relpos_bias_workspace_bytes(2, 4, 100, 90, 32)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    out, g = torch.empty_like(x), torch.zeros(32, 4, device="cuda")

    def both():
        G.relpos_bias(t, out, 128, add=x, q_start=start)
        G.relpos_bias_grad(out, g, ws, 128, q_start=start)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            both()
    torch.cuda.synchronize()
    for k in range(3):
        start.add_(k)
        x.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), g.clone()
        ws.fill_(k)
        both()
        torch.cuda.synchronize()
        assert torch.equal(out, got[0]) and torch.equal(g, got[1])
    with torch.cuda.stream(side):
        both()
    torch.cuda.synchronize()
    assert torch.equal(out, got[0]) and torch.equal(g, got[1])


def line(table, q, k, far, both, start):
    """(heads, q + k - 1): the oracle's bias by diagonal, from j - i = 1 - q on."""
    d = np.arange(1 - q, k) - start
    return torch.from_numpy(f64(table)[O.bucket(d, table.shape[0], far, both)].T.copy()).float().cuda()


def rows_of(lines, q, k, i0, i1):
    """(heads, i1 - i0, k) of the bias."""
    at = torch.arange(k, device="cuda")[None] - torch.arange(i0, i1, device="cuda")[:, None] + q - 1
    return lines[:, at]


@pytest.mark.parametrize("batch,heads,q,k,dtype,shift", [
    (2, 17, 1025, 2112, BF, 0), (2, 17, 1025, 2112, BF, 32), (2, 17, 1025, 2112, BF, 8), (1, 9, 2050, 2080, F32, 16),
    (3, 11, 1030, 2060, BF, 0), (1, 16, 2048, 2048, BF, 0)])
def test_scores_past_the_caches(batch, heads, q, k, dtype, shift):
    """More than 128 MiB and just that, in whole lines and not.  Half-integers and one rounding: exact."""
    rng = np.random.default_rng(k)
    table = torch.from_numpy(rng.integers(-8, 9, (32, heads)) / 2).to(BF).cuda()
    lines = line(table, q, k, 128, True, 3)
    n = batch * heads * q * k
    add = torch.randn(n + 64, device="cuda").to(dtype)[shift:shift + n].view(batch, heads, q, k)
    out = Guarded((batch, heads, q, k), dtype, shift)
    G.relpos_bias(table, out.t, 128, True, q_start=3, add=add)
    out.check()
    want = (add.float() + rows_of(lines, q, k, 0, q)).to(dtype)
    assert torch.equal(out.t, want)
    G.relpos_bias(table, add, 128, True, q_start=3, add=add)
    assert torch.equal(add, want)


@pytest.mark.parametrize("k,shift", [(16384, 0), (16381, 3)])
def test_offsets_past_32_bits(k, shift):
    """Over 2^32 bytes and over 2^31 scores; the gradient's sums are of small whole numbers: exact but
    for the output's rounding."""
    heads, q = 9, 16400
    n = heads * q * k
    assert n > 2 ** 31
    table = torch.from_numpy(np.random.default_rng(k).integers(-8, 9, (32, heads)) / 2).to(BF).cuda()
    lines = line(table, q, k, 128, False, 0)
    add = torch.empty(n + 8, device="cuda", dtype=BF)[shift:shift + n].view(1, heads, q, k)
    add.random_(-2, 3)
    keep = add.clone()
    grad = torch.full((32, heads), 0.5, device="cuda")
    ws = torch.empty(G.relpos_bias_workspace_bytes(1, heads, q, k, 32), dtype=torch.uint8, device="cuda")
    G.relpos_bias_grad(add, grad, ws, 128, False, accumulate=True)
    assert torch.equal(add, keep)
    G.relpos_bias(table, add, 128, False, add=add)
    first = torch.tensor(O.borders(32, 128, False), device="cuda")
    total = torch.zeros(heads, 32, dtype=torch.int64, device="cuda")
    for i in range(0, q, 400):
        to = min(q, i + 400)
        assert torch.equal(add[0, :, i:to], (keep[0, :, i:to].float() + rows_of(lines, q, k, i, to)).to(BF)), i
        # a bucket's columns of a row: distances first[b] to first[b + 1] - 1 to the left, bucket 0 all to the right
        sums = torch.zeros(heads, to - i, k + 1, dtype=torch.int32, device="cuda")
        sums[:, :, 1:] = keep[0, :, i:to].int().cumsum(2, dtype=torch.int32)
        end = (torch.arange(i, to, device="cuda")[:, None] + 1 - first[None]).clamp(0, k)
        end[:, 0] = k
        begin = torch.cat([end[:, 1:], torch.zeros_like(end[:, :1])], 1)
        begin[:, 0] = torch.arange(i, to, device="cuda").clamp(0, k)
        pick = lambda at: sums.gather(2, at[None].expand(heads, -1, -1))  # noqa: E731
        total += (pick(end) - pick(begin)).sum(1)
    assert torch.equal(grad, (total.T + 0.5).float())
