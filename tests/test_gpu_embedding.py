"""Embedding lookup, its gradient and dropout on the GPU against the 64-bit oracle.

Bounds, with u the half step of the output's type (bf16 2^-8, fp32 2^-24) and
e = 2^-24 that of fp32:
  * lookup and dropout without add: the constant is rounded once, the product once,
    the output once: |got - ref| <= |ref| ((1 + e)^2 (1 + u) - 1) + tiny;
  * dropout with add: the product's error (1 + e)^2 - 1 of |x k|, one addition, one
    rounding of the sum;
  * gradient of m terms: a sum of m values in any order is off by at most
    (m - 1) e (1 + e)^m sum|dy|; the constant and the product add 2 e; the old value
    one addition; one rounding.
tiny is half the smallest subnormal of the output's type: 2^-134 (bf16), 2^-150.
"""
import numpy as np
import pytest
import torch

import gradient_sync_zero_amd as G
from oracle import embedding as E
from tests.parity import host

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
EPS = 2.0 ** -24
U = {BF: 2.0 ** -8, F32: EPS}
TINY = {BF: 2.0 ** -134, F32: 2.0 ** -150}
SEED, STEP, SITE = 0x9E3779B97F4A7C15 >> 1, (1 << 32) + 77, 3


def rng_tensor(seed=SEED, step=STEP):
    return torch.tensor([seed, step], dtype=torch.int64, device="cuda")


def f64(t):
    return t.detach().double().cpu().numpy()


class Guarded:
    """A tensor at element `shift` of a longer buffer whose other elements must
    keep their bits."""

    def __init__(self, shape, dtype, shift=0, fill=None):
        n = int(np.prod(shape))
        self.buf = torch.full((n + shift + 24,), 7.25, dtype=dtype, device="cuda")
        self.t = self.buf[shift:shift + n].view(*shape)
        self.lo, self.hi = shift, shift + n
        if fill is not None:
            self.t.copy_(fill)
        else:
            self.t.fill_(float("nan"))

    def check(self):
        assert bool((self.buf[:self.lo] == 7.25).all()) and bool((self.buf[self.hi:] == 7.25).all()), "wrote outside"


def draw(rng, shape, dtype, std=1.0):
    """Values of `dtype` as a device tensor."""
    return torch.from_numpy(rng.normal(0, std, shape).astype(np.float32)).to(dtype).cuda()


def near(got, ref, bound, what):
    got = f64(got)
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3], ref[bad][:3], np.broadcast_to(bound, got.shape)[bad][:3])


def out_bound(ref, dtype, before=2):
    return np.abs(ref) * ((1 + EPS) ** before * (1 + U[dtype]) - 1) + TINY[dtype]


# --------------------------------------------------------------- dropout --

@pytest.mark.parametrize("n", [0, 1, 7, 8, 9, 255, 2047, 2048, 2049, 100_003])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("p,shift", [(0.0, 0), (0.1, 0), (0.5, 1), (0.999, 5)])
def test_dropout(n, dtype, add, p, shift):
    rng = np.random.default_rng(n + 7 * shift)
    x, r = draw(rng, n, dtype), draw(rng, n, dtype)
    gx, gr, gy = Guarded((n,), dtype, shift, x), Guarded((n,), dtype, 3 * shift, r), Guarded((n,), dtype, shift)
    G.dropout(gx.t, gy.t, p, rng_tensor() if p else None, SITE, add=gr.t if add else None)
    for g in (gx, gr, gy):
        g.check()
    scaled = E.dropout(f64(x), p, SEED, STEP, SITE)
    ref = scaled + f64(r) if add else scaled
    bound = out_bound(ref, dtype)
    if add:
        bound = np.abs(scaled) * ((1 + EPS) ** 2 - 1) * (1 + U[dtype]) * (1 + EPS) + out_bound(ref, dtype, 1)
    else:
        assert np.array_equal(f64(gy.t) == 0, ref == 0)
    near(gy.t, ref, bound, "dropout")


@pytest.mark.parametrize("p", [0.1, 2.0 ** -20, 0.5, 0.5 + 2.0 ** -32, 3 * 2.0 ** -17, 1 - 2.0 ** -16, 1 - 2.0 ** -33])
def test_dropout_mask_is_exact_to_32_bits(p):
    """2^22 elements: about 64 of them have the threshold's own high half, so the
    low half decides."""
    n = 1 << 22
    y = torch.empty(n, device="cuda")
    G.dropout(torch.ones(n, device="cuda"), y, p, rng_tensor(), SITE)
    u = E.numbers(0, n, SEED, STEP, SITE)
    assert ((u >> np.uint64(16)) == np.uint64(E.threshold(p) >> 16)).sum() >= 16
    assert np.array_equal(host(y) != 0, u >= np.uint64(E.threshold(p)))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_dropout_in_place_and_backward(dtype):
    n, p = 5003, 0.3
    rng = np.random.default_rng(8)
    x, r = draw(rng, n, dtype), draw(rng, n, dtype)
    want = torch.empty_like(x)
    G.dropout(x, want, p, rng_tensor(), SITE, add=r)
    for keep in ("x", "add"):
        a, b = x.clone(), r.clone()
        G.dropout(a, a if keep == "x" else b, p, rng_tensor(), SITE, add=b)
        assert torch.equal(a if keep == "x" else b, want)
    # the backward pass is the same call: the transpose of a diagonal map is itself
    dx = torch.empty_like(x)
    G.dropout(r, dx, p, rng_tensor(), SITE)
    ref = E.dropout(f64(r), p, SEED, STEP, SITE)
    near(dx, ref, out_bound(ref, dtype), "dx")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_dropped_places_hold_zero_whatever_was_there(dtype):
    n, p = 4096, 0.5
    kept = E.kept(0, n, p, SEED, STEP, SITE)
    for bad in (float("inf"), float("-inf"), float("nan"), torch.finfo(dtype).min):
        x = torch.full((n,), bad, dtype=dtype, device="cuda")
        y = torch.empty_like(x)
        G.dropout(x, y, p, rng_tensor(), SITE)
        got = f64(y)
        assert (got[~kept] == 0).all()
        assert not np.isfinite(got[kept]).any()           # the lowest value doubled overflows


def test_dropout_keeps_subnormals():
    x = torch.tensor([2.0 ** -149 * k for k in range(1, 65)], dtype=torch.float32, device="cuda")
    y = torch.empty_like(x)
    G.dropout(x, y, 0.0, None)
    assert torch.equal(x, y)
    xb = torch.arange(1, 65, dtype=torch.int16).cuda().view(BF)
    yb = torch.empty_like(xb)
    G.dropout(xb, yb, 0.0, None)
    assert torch.equal(xb.view(torch.int16), yb.view(torch.int16))


# ---------------------------------------------------------------- lookup --

@pytest.mark.parametrize("dim", [1, 7, 8, 9, 64, 100, 768, 1531, 8192, 8200, 9001])
@pytest.mark.parametrize("tt,ot,it", [(BF, BF, torch.int64), (BF, F32, torch.int32), (F32, BF, torch.int32),
                                      (F32, F32, torch.int64)])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_lookup(dim, tt, ot, it, p):
    rng = np.random.default_rng(dim)
    for k, n in enumerate((0, 1, 3, 65, 700 if dim < 2000 else 70)):
        rows, shift = (37, 1) if k % 2 else (5000 if dim < 2000 else 60, 0)
        table = Guarded((rows, dim), tt, shift, draw(rng, (rows, dim), tt, 0.02))
        ids = torch.from_numpy(rng.integers(-2, rows + 2, n)).to(it).cuda()
        out = Guarded((n, dim), ot, shift * 3)
        scale = [1.0, float(np.sqrt(dim)), -0.37][k % 3]
        G.embedding_lookup(ids, table.t, out.t, scale=scale, p=p, rng=rng_tensor() if p else None, site=SITE)
        table.check()
        out.check()
        ref = E.lookup(ids.cpu().numpy(), f64(table.t), scale, p, SEED, STEP, SITE)
        assert np.array_equal(f64(out.t) == 0, ref == 0)
        near(out.t, ref, out_bound(ref, ot), (dim, n))


def test_lookup_ids_outside_the_table_give_zero_rows():
    table = torch.full((4, 24), float("nan"), dtype=BF, device="cuda")
    ids = torch.tensor([-1, 4, 1 << 40, -(1 << 40), 1 << 32, (1 << 32) + 1, 2 ** 63 - 1, -2 ** 63], device="cuda")
    out = torch.full((8, 24), 5.0, dtype=BF, device="cuda")
    G.embedding_lookup(ids, table, out)
    assert bool((out == 0).all())
    i32 = torch.tensor([-1, 4, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    out.fill_(5.0)
    G.embedding_lookup(i32, table, out[:4])
    assert bool((out[:4] == 0).all()) and bool((out[4:] == 5).all())
    none = torch.empty(0, 24, dtype=BF, device="cuda")          # a table without rows
    out.fill_(5.0)
    G.embedding_lookup(ids, none, out)
    assert bool((out == 0).all())


def test_lookup_with_dropout_has_the_mask_of_dropout():
    ids, table = torch.arange(50, device="cuda") % 7, torch.randn(7, 333, device="cuda")
    a, b, c = (torch.empty(50, 333, device="cuda") for _ in range(3))
    G.embedding_lookup(ids, table, a, p=0.2, rng=rng_tensor(), site=SITE)
    G.embedding_lookup(ids, table, b)
    G.dropout(b, c, 0.2, rng_tensor(), SITE)
    assert torch.equal(a, c)


# -------------------------------------------------------------- gradient --

def make_ids(kind, n, rows, rng):
    if kind == "one":
        ids = np.full(n, rows // 2)
    elif kind == "hot":
        ids = np.where(rng.random(n) < 0.9, rows // 3, rng.integers(0, rows, n))
    elif kind == "none":
        ids = np.where(rng.random(n) < 0.5, -1, rows)
    elif kind == "distinct":
        ids = np.arange(n) % rows
    elif kind == "falling":
        ids = (rows - 1 - np.arange(n) * 3 // 7) % rows
    else:
        ids = rng.integers(-1, rows + 1, n)
    return ids.astype(np.int64)


def run_grad(ids, dy, grad, **kw):
    n, (rows, dim) = ids.numel(), grad.shape
    ws = torch.full((G.embedding_workspace_bytes(n, rows, dim) // 4 + 4,), float("nan"), device="cuda")
    ws[-4:] = 7.25
    G.embedding_grad(ids, dy, grad, ws[:-4], **kw)
    assert bool((ws[-4:] == 7.25).all()), "wrote past the workspace"


def check_grad(n, rows, dim, kind="any", dt=BF, gt=BF, it=torch.int64, acc=False, p=0.0, scale=1.0, shift=0, seed=0):
    rng = np.random.default_rng(seed + n + rows + dim)
    ids = torch.from_numpy(make_ids(kind, n, rows, rng)).to(it).cuda()
    dy = Guarded((n, dim), dt, shift, draw(rng, (n, dim), dt))
    old = draw(rng, (rows, dim), gt) if acc else None
    g = Guarded((rows, dim), gt, 3 * shift, old)
    kw = dict(scale=scale, p=p, rng=rng_tensor() if p else None, site=SITE, accumulate=acc)
    run_grad(ids, dy.t, g.t, **kw)
    g.check()
    dy.check()
    i = ids.cpu().numpy()
    ref, size = E.grad(i, f64(dy.t), rows, scale, p, SEED, STEP, SITE, None if old is None else f64(old))
    m = np.bincount(i[(i >= 0) & (i < rows)], minlength=rows).astype(float)[:, None]
    summed = size * ((1 + EPS) ** (m + 3) - 1)
    bound = summed * (1 + U[gt]) * (1 + EPS) + out_bound(ref, gt, 1)
    near(g.t, ref, bound, (n, rows, dim, kind))
    # rows without a token: exactly the old bits, or exactly zero
    rest = torch.from_numpy(m[:, 0] == 0).cuda()
    assert torch.equal(g.t[rest], old[rest]) if acc else bool((g.t[rest] == 0).all())
    # the same call once more gives the same bits
    again = Guarded((rows, dim), gt, 3 * shift, old)
    run_grad(ids, dy.t, again.t, **kw)
    assert torch.equal(again.t, g.t)


@pytest.mark.parametrize("n", [0, 1, 2, 5, 63, 64, 65, 127, 128, 129, 200, 511])
@pytest.mark.parametrize("kind", ["any", "one", "none", "distinct"])
@pytest.mark.parametrize("acc", [False, True])
def test_grad_small(n, kind, acc):
    check_grad(n, 100, 40, kind, acc=acc, gt=F32 if n % 2 else BF, dt=BF if n % 3 else F32)


@pytest.mark.parametrize("dim", [1, 7, 8, 9, 100, 511, 512, 513, 768, 1531, 2056, 4097])
@pytest.mark.parametrize("dt,gt,it", [(BF, BF, torch.int64), (BF, F32, torch.int32), (F32, BF, torch.int64),
                                      (F32, F32, torch.int32)])
@pytest.mark.parametrize("acc,p,shift", [(False, 0.0, 0), (True, 0.25, 1)])
def test_grad_widths_and_types(dim, dt, gt, it, acc, p, shift):
    check_grad(300, 90, dim, "hot", dt, gt, it, acc, p, float(np.sqrt(dim)), shift)


@pytest.mark.parametrize("n", [8191, 8192, 8193, 9000, 20_000, 66_000])
@pytest.mark.parametrize("kind", ["any", "one", "hot", "falling", "none"])
def test_grad_many_tokens(n, kind):
    """Both sorts and every level of the joining of long runs."""
    check_grad(n, 5000, 24, kind, BF, F32, acc=n % 2 == 0)


@pytest.mark.parametrize("n", [1, 5, 64, 128, 129, 700, 9000])
@pytest.mark.parametrize("dim", [40, 41, 520])
@pytest.mark.parametrize("dt", [BF, F32])
def test_grad_with_dropout_on_every_path(n, dim, dt):
    check_grad(n, 60, dim, "any", dt, F32, acc=n % 2 == 0, p=0.3, scale=0.5, shift=n % 3)
    check_grad(n, 60, dim, "one", dt, BF, acc=n % 2 == 1, p=0.7)


@pytest.mark.parametrize("dt,gt", [(BF, BF), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("dim,kind", [(2048, "any"), (2051, "hot")])
@pytest.mark.parametrize("acc", [False, True])
def test_grad_of_large_dy(dt, gt, dim, kind, acc):
    """dy of over 64 MiB, which is read nontemporally, against torch in 64 bits."""
    n, rows = 18_000, 3000
    rng = np.random.default_rng(dim)
    ids = torch.from_numpy(make_ids(kind, n, rows, rng)).cuda()
    gen = torch.Generator(device="cuda").manual_seed(dim)
    dy = torch.randn(n, dim, device="cuda", generator=gen).to(dt)
    old = torch.randn(rows, dim, device="cuda", generator=gen).to(gt)
    grad = old.clone() if acc else torch.full_like(old, float("nan"))
    run_grad(ids, dy, grad, scale=3.0, accumulate=acc)
    ok = (ids >= 0) & (ids < rows)
    ref = torch.zeros(rows, dim, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(ref)
    ref.index_add_(0, ids[ok], dy[ok].double())
    size.index_add_(0, ids[ok], dy[ok].double().abs())
    ref, size = ref * 3 + (old.double() if acc else 0), size * 3
    m = torch.bincount(ids[ok], minlength=rows).double()[:, None]
    # torch's own 64-bit sums are off by at most m 2^-53 of size: far below EPS size
    bound = size * ((1 + EPS) ** (m + 4) - 1) * (1 + U[gt]) * (1 + EPS) + ref.abs() * ((1 + EPS) * (1 + U[gt]) - 1) + TINY[gt]
    assert bool(((grad.double() - ref).abs() <= bound).all())


@pytest.mark.parametrize("rows", [0, 1, 2, 255, 256, 1023, 1024, 70_000, (1 << 20) - 1, 1 << 20, 1_100_003])
def test_grad_table_heights(rows):
    """One to three passes of the counting sort, keys at the digits' borders."""
    check_grad(8300, rows, 8, "any", BF, BF)
    check_grad(100, rows, 8, "any", BF, F32, acc=True)


def test_grad_four_sort_passes_and_tall_table():
    rows, n = (1 << 30) + 5, 9000
    rng = np.random.default_rng(1)
    ids = rng.integers(0, rows, n)
    ids[:7] = [rows - 1, 0, rows - 1, 1 << 30, (1 << 29) + 1, rows, -1]
    dy = draw(rng, (n, 1), F32)
    grad = torch.zeros(rows, 1, dtype=F32, device="cuda")
    run_grad(torch.from_numpy(ids).cuda(), dy, grad, accumulate=True)
    ok = (ids >= 0) & (ids < rows)
    at, back = np.unique(ids[ok], return_inverse=True)
    ref = np.zeros(at.size)
    np.add.at(ref, back, f64(dy)[ok, 0])
    got = f64(grad[torch.from_numpy(at).cuda(), 0])
    assert np.abs(got - ref).max() <= 64 * EPS * np.abs(f64(dy)).max() * 3
    assert int((grad != 0).sum()) <= at.size


def test_grad_tiles_of_the_sort_grow():
    check_grad(300_001, 700, 4, "any", BF, F32)            # over 256 tiles of 1024


def test_grad_masked_places_and_bad_values():
    """An infinity or NaN in a dropped place or at a token without a row leaves
    no trace; one that counts reaches its own row only."""
    n, rows, dim, p = 600, 20, 64, 0.5
    kept = E.kept(0, n * dim, p, SEED, STEP, SITE).reshape(n, dim)
    rng = np.random.default_rng(3)
    ids = rng.integers(0, rows - 1, n)
    ids[::5] = -1
    dy = rng.normal(size=(n, dim)).astype(np.float32)
    bad = np.where(rng.random((n, dim)) < 0.5, np.inf, np.nan).astype(np.float32)
    masked = np.where(kept & (ids >= 0)[:, None], dy, bad)
    g = [torch.empty(rows, dim, device="cuda") for _ in range(2)]
    kw = dict(p=p, rng=rng_tensor(), site=SITE)
    for t, v in zip(g, (dy, masked)):
        run_grad(torch.from_numpy(ids).cuda(), torch.from_numpy(v).cuda(), t, **kw)
    assert torch.equal(g[0], g[1]) and bool(torch.isfinite(g[0]).all())
    i = int(np.flatnonzero(ids == 4)[0])
    dy[i] = np.inf
    run_grad(torch.from_numpy(ids).cuda(), torch.from_numpy(dy).cuda(), g[1], **kw)
    rest = torch.arange(rows, device="cuda") != 4
    assert torch.equal(g[0][rest], g[1][rest])
    assert np.array_equal(np.isinf(f64(g[1][4])), kept[i])


def test_grad_is_the_derivative_of_the_lookup_by_differences():
    """<dy, lookup(table + d) - lookup(table)> = <grad, d> in values that the sums
    hold exactly (small integers), so the two sides are equal."""
    rng = np.random.default_rng(12)
    rows, dim, n = 40, 96, 500
    ids = torch.from_numpy(rng.integers(-1, rows + 1, n)).cuda()
    whole = lambda *s: torch.from_numpy(rng.integers(-4, 5, s).astype(np.float32)).cuda()
    table, d, dy = whole(rows, dim), whole(rows, dim), whole(n, dim)
    kw = dict(scale=2.0, p=0.5, rng=rng_tensor(), site=SITE)
    a, b, g = torch.empty(n, dim, device="cuda"), torch.empty(n, dim, device="cuda"), torch.empty(rows, dim, device="cuda")
    G.embedding_lookup(ids, table, a, **kw)
    G.embedding_lookup(ids, table + d, b, **kw)
    run_grad(ids, dy, g, **kw)
    assert ((b - a).double() * dy.double()).sum() == (g.double() * d.double()).sum()


# ------------------------------------------------- streams, graphs, sizes --

def test_on_another_stream():
    side = torch.cuda.Stream()
    rng = np.random.default_rng(2)
    ids = torch.from_numpy(rng.integers(0, 50, 9000)).cuda()
    dy = draw(rng, (9000, 64), BF)
    outs = []
    torch.cuda.synchronize()
    for st in (None, side, side.cuda_stream):
        table, out, grad, y = draw(np.random.default_rng(5), (50, 64), BF), torch.empty_like(dy), torch.empty(50, 64, device="cuda"), torch.empty_like(dy)
        ws = torch.empty(G.embedding_workspace_bytes(9000, 50, 64), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        G.embedding_lookup(ids, table, out, p=0.1, rng=rng_tensor(), stream=st)
        G.dropout(out, y, 0.2, rng_tensor(), 1, add=dy, stream=st)
        G.embedding_grad(ids, y, grad, ws, p=0.1, rng=rng_tensor(), stream=st)
        torch.cuda.synchronize()
        outs.append((out, y, grad))
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))


def test_two_calls_at_once():
    """Two gradients on two streams with a workspace each, over and over, have the
    bits that each has alone."""
    rng = np.random.default_rng(31)
    rows, dim = 4000, 512
    cases = []
    for n in (9000, 3000):
        ids, dy = torch.from_numpy(make_ids("hot", n, rows, rng)).cuda(), draw(rng, (n, dim), BF)
        alone = torch.empty(rows, dim, device="cuda")
        run_grad(ids, dy, alone)
        ws = torch.empty(G.embedding_workspace_bytes(n, rows, dim), dtype=torch.uint8, device="cuda")
        cases.append((ids, dy, ws, alone, torch.cuda.Stream(), [torch.empty_like(alone) for _ in range(5)]))
    torch.cuda.synchronize()
    for k in range(5):
        for ids, dy, ws, _, st, outs in cases:
            G.embedding_grad(ids, dy, outs[k], ws, stream=st)
    torch.cuda.synchronize()
    for *_, alone, _, outs in cases:
        assert all(torch.equal(o, alone) for o in outs)


@pytest.mark.parametrize("n", [300, 9000])
def test_graph_replays_equal_eager_calls(n):
    """Captured once, replayed with other tokens and another step in the same
    memory: each replay has the eager call's bits and a mask of its own."""
    rows, dim, p = 200, 776, 0.1
    rng = np.random.default_rng(n)
    ids = torch.zeros(n, dtype=torch.int64, device="cuda")
    key = rng_tensor()
    table = draw(rng, (rows, dim), BF)
    ws = torch.empty(G.embedding_workspace_bytes(n, rows, dim), dtype=torch.uint8, device="cuda")

    def buffers():
        return dict(out=torch.empty(n, dim, dtype=BF, device="cuda"), y=torch.empty(n, dim, dtype=BF, device="cuda"),
                    dx=torch.empty(n, dim, dtype=BF, device="cuda"), acc=torch.ones(rows, dim, device="cuda"),
                    g=torch.full((rows, dim), 9.0, dtype=BF, device="cuda"))

    def step(b):
        G.embedding_lookup(ids, table, b["out"], scale=3.0, p=p, rng=key, site=0)
        G.dropout(b["out"], b["y"], p, key, 1, add=b["out"])
        G.dropout(b["y"], b["dx"], p, key, 1)
        G.embedding_grad(ids, b["dx"], b["acc"], ws, scale=3.0, p=p, rng=key, site=0, accumulate=True)
        G.embedding_grad(ids, b["dx"], b["g"], ws, scale=3.0, p=p, rng=key, site=0)

    eager, b = buffers(), buffers()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        step(b)
    seen = []
    for k in range(4):
        ids.copy_(torch.from_numpy(make_ids(["any", "hot", "one", "none"][k], n, rows, rng)).cuda())
        key.copy_(rng_tensor(step=k))
        step(eager)
        torch.cuda.synchronize()
        graph.replay()
        junk = torch.randn(1 << 20, device="cuda").sum()
        torch.cuda.synchronize()
        for name in b:
            assert torch.equal(b[name], eager[name]), (k, name)
        seen.append((b["y"] == b["out"]).clone())
        del junk
    assert all(not torch.equal(seen[i], seen[j]) for i in range(3) for j in range(i))


def test_offsets_past_32_bits():
    """n * dim and rows * dim of over 2^32 values: the far ends against torch on
    the rows concerned."""
    n, dim, rows = 70_000, 65_544, 66_000
    ids = (torch.arange(n, device="cuda") * 7919) % rows
    table = torch.zeros(rows, dim, dtype=BF, device="cuda")
    pick = torch.tensor([0, 1, 65_535, 65_536, rows - 1], device="cuda")
    table[pick] = torch.randn(5, dim, device="cuda").to(BF)
    out = torch.full((n, dim), 3.0, dtype=BF, device="cuda")
    G.embedding_lookup(ids, table, out, scale=2.0)
    for i in (0, 1, 65_535, 65_536, 69_999) + tuple(int(x) for v in pick for x in (ids == v).nonzero()[:, 0]):
        assert torch.equal(out[i], table[ids[i]] * 2)
    del table
    # masks far out: element (n - 1) * dim + c
    G.dropout(out.view(-1), out.view(-1), 0.5, rng_tensor(), SITE)
    first = (n - 1) * dim
    assert np.array_equal(f64(out[n - 1]) == 0, ~E.kept(first, dim, 0.5, SEED, STEP, SITE) | (f64(out[n - 1]) == 0))
    assert (f64(out[n - 1])[~E.kept(first, dim, 0.5, SEED, STEP, SITE)] == 0).all()
    dy = out
    dy.fill_(1.0)
    dy[n - 1] = 5.0
    grad = torch.full((rows, dim), 9.0, dtype=BF, device="cuda")
    run_grad(ids, dy, grad, p=0.5, rng=rng_tensor(), site=SITE)
    v = int(ids[n - 1])
    ref = torch.zeros(dim, dtype=torch.float64)
    for i in (ids == v).nonzero()[:, 0].tolist():
        kept = torch.from_numpy(E.kept(i * dim, dim, 0.5, SEED, STEP, SITE))
        ref += torch.where(kept, dy[i].double().cpu() * 2, 0.0)
    assert torch.equal(grad[v].double().cpu(), ref)
    assert bool((grad[torch.arange(rows, device="cuda")[torch.bincount(ids, minlength=rows) == 0]] == 0).all())


def test_refuses_tensors_of_host_and_bad_workspace():
    ids, dy = torch.zeros(200, dtype=torch.int64, device="cuda"), torch.zeros(200, 8, dtype=BF, device="cuda")
    grad = torch.zeros(3, 8, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="device tensor"):
        G.embedding_lookup(ids.cpu(), grad, dy)
    with pytest.raises(ValueError, match="contiguous"):
        G.embedding_lookup(ids, torch.zeros(8, 3, dtype=BF, device="cuda").t(), dy)
    with pytest.raises(G.GszError) as e:
        G.embedding_grad(ids, dy, grad, torch.empty(8, device="cuda"))
    assert e.value.name == "GSZ_ERR_SIZE"
    with pytest.raises(G.GszError) as e:
        G.embedding_grad(ids, dy, grad, None)
    assert e.value.name == "GSZ_ERR_SIZE"
    with pytest.raises(G.GszError) as e:
        G.dropout(dy, dy, 0.1, None)
    assert e.value.name == "GSZ_ERR_INVALID_ARG"
