"""Newton-Schulz orthogonalisation and the Muon update on the GPU against the 64-bit oracle.

Bounds (2-norm over a matrix), u = 2^-8 the half step of bf16:
  * against the exact result: oracle.muon.rounding_bound, what rounding X, A and S to fp16 can do
    to first order, doubled for the rest and for the fp32 sums; and u |O| for the output;
  * against the oracle with the same roundings: the kernel's fp32 sums differ from 64-bit ones by
    up to about K 2^-24 of the terms, so a rounding goes the other way where a value lies that close
    to a tie: of K <= 2^11 terms of random sign, about sqrt(K) 2^-24 / 2^-11 < 2^-7 of the values move
    by a step 2^-10, 2^-10 sqrt(2^-7) < 9e-5 of the norm for each of the 15 roundings (17 where steps go
    in pairs), grown by at most
    3.5 a step (sum over steps of 3 * 3.5^(4 - k) < 630 in the first order's worst case, about 10 where
    the change is spread over all directions): 1e-3 for the fp32 result; for bf16 1e-3 of change
    moves 1e-3 / 2^-8 < 26% of the roundings by 2^-7 at most: sqrt(0.26) 2^-8 < 2e-3 more.
"""
import numpy as np
import pytest
import torch

import gradient_sync_zero_amd as G
from oracle import muon as O
from tests.parity import host

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -8


def f64(t):
    return t.detach().double().cpu().numpy()


def norm(x):
    return float(np.sqrt((np.asarray(x, dtype=np.float64) ** 2).sum()))


def workspace(count, rows, cols, fill=0xFF):
    return torch.full((G.muon_workspace_bytes(count, rows, cols) + 16,), fill, dtype=torch.uint8, device="cuda")


def run(x, **kw):
    """orthogonalize into a guarded buffer, from a workspace of NaNs of just the documented size."""
    count = 1 if x.dim() == 2 else x.shape[0]
    ws = workspace(count, *x.shape[-2:])
    buf = torch.full((x.numel() + 48,), 7.25, dtype=BF, device="cuda")
    out = buf[24:24 + x.numel()].view(x.shape)
    before = x.clone()
    G.orthogonalize(x, out, ws[:-16], **kw)
    assert bool((buf[:24] == 7.25).all()) and bool((buf[-24:] == 7.25).all()), "wrote outside"
    assert bool((ws[-16:] == 0xFF).all()), "wrote behind the workspace"
    assert torch.equal(x, before)
    return out


def check(out, x, count=None, **kw):
    """count: how many matrices the call had, where out and x are only some of them."""
    count = count or (1 if x.dim() == 2 else x.shape[0])
    for got, xi in zip(f64(out).reshape(-1, *out.shape[-2:]), f64(x).reshape(-1, *x.shape[-2:])):
        exact, same = O.orthogonalize(xi, **kw), O.orthogonalize(xi, rounded=True, count=count, **kw)
        d = norm(got - exact)
        assert d <= 2 * O.rounding_bound(xi, **kw) + U * norm(exact), d / norm(exact)
        d = norm(got - same.astype(np.float32))
        assert d <= (3e-3 + U) * norm(same), d / norm(same)


SHAPES = [(1, 1), (1, 7), (5, 1), (2, 3), (17, 64), (64, 17), (63, 65), (128, 128), (129, 127), (1, 3001), (200, 500),
          (500, 200), (300, 300), (257, 1000), (33, 2049), (128, 256), (256, 128), (128, 257), (257, 128), (129, 129), (96, 160), (2049, 97)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_matrix(rows, cols, dtype):
    x = torch.from_numpy(np.random.default_rng(rows * 7 + cols).normal(0, 1e-3, (rows, cols))).to(dtype).cuda()
    check(run(x), x)


@pytest.mark.parametrize("count,rows,cols", [(3, 40, 90), (260, 20, 9), (50, 300, 257), (210, 130, 60), (30, 768, 200)])
def test_many_matrices(count, rows, cols):
    """Several a launch, more than one launch holds (256), and enough for the large tiles."""
    rng = np.random.default_rng(count)
    x = torch.from_numpy(rng.normal(0, 1, (count, rows, cols)) * 10.0 ** rng.uniform(-6, 6, (count, 1, 1))).to(F32).cuda()
    out = run(x)
    some = [0, 1, count // 2, count - 2, count - 1]
    check(out[some], x[some], count)
    # each by itself gives the same bits
    for b in some[::2]:
        assert torch.equal(run(x[b]), out[b])


@pytest.mark.parametrize("count,rows,cols", [(1, 1100, 2300), (9, 1030, 640), (20, 900, 520), (2, 2100, 2000), (26, 64, 3001), (150, 700, 90),
                                             (3, 200, 1700), (2, 1700, 150), (1, 600, 2000), (1, 1990, 610), (1, 2300, 3700),
                                             (12, 400, 1100), (25, 1400, 900)])
def test_large(count, rows, cols):
    """Every size of tiles, last rounds that are cut along the sums, and panels of several matrices."""
    rng = np.random.default_rng(rows)
    x = torch.from_numpy(rng.normal(0, 1, (count, rows, cols))).to(F32).cuda()
    out = run(x)
    check(out[[0, count - 1]], x[[0, count - 1]], count)


def test_low_rank_and_wide_spectrum():
    rng = np.random.default_rng(4)
    for s in (np.r_[1.0, np.zeros(59)], 10.0 ** -np.linspace(0, 3, 60)):
        u, v = np.linalg.qr(rng.normal(size=(60, 60)))[0], np.linalg.qr(rng.normal(size=(100, 60)))[0]
        x = torch.from_numpy((u * s) @ v.T).to(F32).cuda()
        out = run(x)
        exact = O.orthogonalize(f64(x))
        assert norm(f64(out) - exact) <= 2 * O.rounding_bound(f64(x)) + U * norm(exact)


@pytest.mark.parametrize("steps", [1, 2, 3, 6, 16])
def test_steps_and_coefficients(steps):
    x = torch.from_numpy(np.random.default_rng(steps).normal(size=(70, 150))).to(F32).cuda()
    check(run(x, steps=steps), x, steps=steps)
    ns = [(1.5, -0.5, 0.0)] * (steps - 1) + [(1.875, -1.25, 0.375)]
    check(run(x, steps=steps, ns=ns), x, steps=steps, ns=ns)


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 6, 7])
def test_pairs_of_steps(steps):
    """Long matrices take two steps at once, of an odd number one alone."""
    assert O.in_pairs(140, 1200) and O.in_pairs(1400, 170) and O.in_pairs(400, 1100, 12) and O.in_pairs(1400, 900, 25)
    assert not (O.in_pairs(400, 1100) or O.in_pairs(1400, 900))
    for rows, cols in ((140, 1200), (1400, 170)):
        x = torch.from_numpy(np.random.default_rng(steps).normal(size=(2, rows, cols))).to(F32).cuda()
        ns = [(1.5, -0.5, 0.0), (1.875, -1.25, 0.375)] * 4
        check(run(x, steps=steps, ns=ns[:steps]), x, steps=steps, ns=ns[:steps])
        check(run(x, steps=steps), x, steps=steps)


def test_scale_of_the_input_does_not_matter_and_eps_does():
    x = torch.from_numpy(np.random.default_rng(5).normal(size=(40, 60))).to(F32).cuda()
    want = run(x, eps=1e-30)
    for e in (-60, 40):                                   # powers of two: the same bits
        assert torch.equal(run(x * 2.0 ** e, eps=1e-30), want)
    check(run(x * 1e-6, eps=1e-4), x * 1e-6, eps=1e-4)
    big = torch.full((8, 8), 3e38, device="cuda")         # squares far past fp32's range
    check(run(big), big)


def test_zeros_and_values_that_are_not_finite():
    x = torch.from_numpy(np.random.default_rng(6).normal(size=(5, 30, 50))).to(F32).cuda()
    want = run(x)
    x[1] = 0.0
    x[3, 4, 5] = float("inf")
    x[4, 0, 0] = float("nan")
    out = run_keep(x)
    assert bool((out[1] == 0).all()) and bool(out[3:].isnan().all())
    assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2])


def run_keep(x):
    out = torch.empty(x.shape, dtype=BF, device="cuda")
    G.orthogonalize(x, out, workspace(x.shape[0], *x.shape[1:]))
    return out


def test_in_place_and_unaligned():
    x = torch.from_numpy(np.random.default_rng(7).normal(size=(2, 37, 51))).to(BF).cuda()
    want = run(x)
    for shift in (0, 1, 3, 8):
        buf = torch.empty(x.numel() + 8, dtype=BF, device="cuda")
        y = buf[shift:shift + x.numel()].view(x.shape)
        y.copy_(x)
        G.orthogonalize(y, y, workspace(2, 37, 51))
        assert torch.equal(y, want)
        z = torch.empty(x.numel() + 8, dtype=F32, device="cuda")[shift:shift + x.numel()].view(x.shape)
        z.copy_(x)
        G.orthogonalize(z, y, workspace(2, 37, 51))
        assert torch.equal(y, want)


def test_empty():
    for shape in ((0, 3, 4), (2, 0, 4), (2, 3, 0)):
        G.orthogonalize(torch.empty(shape, device="cuda"), torch.empty(shape, dtype=BF, device="cuda"), None)


# ------------------------------------------------------------------- update --

LR, MU, WD = 0.02, 0.95, 0.1


def flats(plan, rng, odd=0.0):
    mk = lambda s: torch.from_numpy(rng.normal(0, s, plan.flat_len).astype(np.float32)).cuda()  # noqa: E731
    return mk(0.02), mk(4e-3), mk(1e-3), torch.full((plan.flat_len,), 0x7777, dtype=torch.uint16, device="cuda")


@pytest.mark.parametrize("rows,cols,numel,tensors", [
    (64, 96, [6144, 37, 6144, 6144], [0, 3, 2]), (300, 130, [39000, 1], [0]), (1, 9, [9, 9, 9, 100], [2, 0]),
    (130, 300, [5, 39000, 7, 39000], [3, 1]), (16, 16, [256] * 300, list(range(299, -1, -1)))])
@pytest.mark.parametrize("nesterov", [True, False])
def test_update(rows, cols, numel, tensors, nesterov):
    rng = np.random.default_rng(rows + cols)
    plan = G.Plan(numel, 1 << 16, 4)
    w, m, g, p = flats(plan, rng)
    w0, m0, g0 = host(w).copy(), host(m).copy(), host(g)
    coef = torch.tensor([0.37], device="cuda")
    scale = 0.2 * max(rows, cols) ** 0.5
    hp = G.make_muon_hp(lr=LR, momentum=MU, weight_decay=WD, scale=scale, nesterov=nesterov)
    G.muon_step(plan, tensors, rows, cols, w, m, g, coef, hp, p, workspace(len(tensors), rows, cols))
    assert torch.equal(g, torch.from_numpy(g0).cuda())
    p16 = host(p)
    touched = np.zeros(plan.flat_len, dtype=bool)
    w1, m1 = host(w), host(m)
    f = np.float32
    for t in tensors:
        s = slice(plan.tensor(t)[0], plan.tensor(t)[0] + rows * cols)
        touched[s] = True
        # the momentum in the library's order of roundings: bit for bit
        gc = g0[s] * f(host(coef)[0])
        want = f(MU) * m0[s] + gc
        assert np.array_equal(m1[s], want)
        if t in tensors[:3] + tensors[-3:]:
            u = (gc + f(MU) * want if nesterov else want).reshape(rows, cols)
            same = O.orthogonalize(u, rounded=True, count=len(tensors))
            exact = O.orthogonalize(u)
            got = (w0[s].astype(np.float64) * float(f(1 - LR * WD)) - w1[s]).reshape(rows, cols) / float(f(LR * scale))
            # the update's own roundings: theta to fp32 three times, 2^-24 of it each
            slack = 3 * 2.0 ** -24 * norm(w0[s]) / (LR * scale)
            assert norm(got - same) <= 1e-3 * norm(same) + slack
            assert norm(got - exact) <= 2 * O.rounding_bound(u) + slack
    assert np.array_equal(w1[~touched], w0[~touched]) and np.array_equal(m1[~touched], m0[~touched])
    assert bool((p16[~touched] == 0x7777).all())
    assert np.array_equal(p16[touched], host(w.bfloat16().view(torch.uint16))[touched])


def test_update_matches_orthogonalize_of_the_same_direction():
    plan = G.Plan([100 * 60], 1 << 40, 1)
    w, m, g, p = flats(plan, np.random.default_rng(2))
    w.zero_()
    coef = torch.ones(1, device="cuda")
    hp = G.make_muon_hp(lr=1.0, momentum=0.0, scale=-1.0, nesterov=False)
    G.muon_step(plan, [0], 100, 60, w, m, g, coef, hp, p, workspace(1, 100, 60))
    out = torch.empty(100, 60, dtype=BF, device="cuda")
    G.orthogonalize(plan.view(0, g).view(100, 60), out, workspace(1, 100, 60))
    assert torch.equal(plan.view(0, p).view(torch.bfloat16), out.view(-1))


def test_capture_and_other_streams():
    """A captured update replayed with the program's own work between, and two calls at once on
    two streams with a workspace each, give the eager result."""
    rows, cols = 150, 90
    plan = G.Plan([rows * cols] * 3, 1 << 40, 1)
    rng = np.random.default_rng(11)
    w, m, g, p = flats(plan, rng)
    coef = torch.tensor([0.5], device="cuda")
    hp = G.make_muon_hp(lr=LR, scale=2.0, weight_decay=WD)
    ws = workspace(3, rows, cols)
    start = [t.clone() for t in (w, m, p)]
    want = []
    for _ in range(3):
        G.muon_step(plan, [0, 1, 2], rows, cols, w, m, g, coef, hp, p, ws)
        want.append([t.clone() for t in (w, m, p)])
    for t, s in zip((w, m, p), start):
        t.copy_(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            G.muon_step(plan, [0, 1, 2], rows, cols, w, m, g, coef, hp, p, ws)
    torch.cuda.synchronize()
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        ws.fill_(k)                                          # nothing is kept there between calls
        for t, s in zip((w, m, p), want[k]):
            assert torch.equal(t, s), k
    x = torch.from_numpy(rng.normal(size=(2, 4, rows, cols))).to(F32).cuda()
    alone = [run_keep(x[k]) for k in range(2)]
    outs = [torch.empty(x[0].shape, dtype=BF, device="cuda") for _ in range(2)]
    spaces = [workspace(4, rows, cols) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for k in range(2):
            G.orthogonalize(x[k], outs[k], spaces[k], stream=streams[k])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], alone[0]) and torch.equal(outs[1], alone[1])


@pytest.mark.parametrize("rows,cols", [(2 ** 17, 16400), (16400, 2 ** 17)])
def test_offsets_past_32_bits(rows, cols):
    """Over 2^31 elements and 2^32 bytes: signs (-1)^popcount(i & j), whose columns (rows) are orthogonal,
    so that every singular value is the same and the result is x times a number, f(f(f(f(f(s))))).
    A rounding, off by h = 2^-11, of X, A or S (three a step, in pairs fewer than four) changes a
    step's result by at most h (|a| s + 3 |b| s^3 + 5 |c| s^5), and the later steps that by s f'/f
    each; doubled for what lies beyond the first order, and u for the output."""
    n, m = max(rows, cols), min(rows, cols)
    assert rows * cols > 2 ** 31

    def signs(i0, i1):
        v = torch.arange(i0, i1, device="cuda", dtype=torch.int32)[:, None] & torch.arange(cols, device="cuda", dtype=torch.int32)[None]
        for shift in (16, 8, 4, 2, 1):
            v = v ^ (v >> shift)
        return (1 - 2 * (v & 1)).to(BF)

    x = torch.empty(rows, cols, dtype=BF, device="cuda")
    step = 2 ** 26 // cols
    for i in range(0, rows, step):
        x[i:i + step] = signs(i, min(rows, i + step))
    ws = torch.empty(G.muon_workspace_bytes(1, rows, cols), dtype=torch.uint8, device="cuda")
    G.orthogonalize(x, x, ws)
    a, b, c = O.NS
    s, off = m ** -0.5, 0.0
    for _ in range(5):
        f = a * s + b * s ** 3 + c * s ** 5
        off = off * abs(s * (a + 3 * b * s ** 2 + 5 * c * s ** 4) / f) + 4 * 2.0 ** -11 * (a * s + 3 * abs(b) * s ** 3 + 5 * c * s ** 5) / abs(f)
        s = f
    want = s * n ** -0.5
    for i in range(0, rows, step):
        got = x[i:i + step].float() * signs(i, min(rows, i + step)).float() / want
        assert float((got - 1).abs().max()) <= 2 * off + U, (i, 2 * off)
