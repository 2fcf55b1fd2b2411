"""Host-side checks of the orthogonalising update and the relative position bias: what they
refuse before any device call, through the C ABI and through the binding."""
import ctypes
import os
import re

import pytest

import gradient_sync_zero_amd as G
from tests.test_layers_cpu import Dev

BF16, F32, I32, I64 = 0, 1, 2, 3
INVALID, MISALIGNED, SIZE = -1, -2, -3
BUF, APART = 1 << 20, 1 << 40           # aligned addresses that no refused call reads
NAN, INF = float("nan"), float("inf")


def orth(lib, x=BUF, t=BF16, count=2, rows=6, cols=8, steps=5, ns=None, eps=1e-7, out=APART, ws=2 * APART, ws_bytes=1 << 40):
    arr = None if ns is None else (ctypes.c_double * len(ns))(*ns)
    return lib.gsz_orthogonalize(x, t, count, rows, cols, steps, arr, eps, out, ws, ws_bytes, None)


def muon(lib, numel=(48, 5, 48), tensors=(0, 2), count=None, rows=6, cols=8, w=BUF, m=APART, g=2 * APART, coef=3 * APART, p=4 * APART,
         ws=5 * APART, ws_bytes=1 << 39, no_plan=False, no_hp=False, no_list=False, **hp):
    plan = G.Plan(list(numel), 1 << 20, 2)
    arr = None if no_list else (ctypes.c_int32 * max(len(tensors), 1))(*tensors)
    h = G.make_muon_hp(**dict(dict(lr=0.1), **hp))
    return lib.gsz_muon_step(None if no_plan else plan.handle, arr, len(tensors) if count is None else count, rows, cols, w, m, g, coef,
                             None if no_hp else ctypes.byref(h), p, ws, ws_bytes, None)


def bias(lib, table=BUF, tt=BF16, buckets=32, heads=2, far=128, both=1, batch=1, q=3, k=4, start=0, starts=None, st=I64, scale=1.0,
         add=None, out=APART, ot=BF16):
    return lib.gsz_relpos_bias(table, tt, buckets, heads, far, both, batch, q, k, start, starts, st, scale, add, out, ot, None)


def grad(lib, dy=BUF, dt=BF16, buckets=32, heads=2, far=128, both=1, batch=1, q=3, k=4, start=0, starts=None, st=I64, scale=1.0,
         g=APART, gt=F32, acc=0, ws=2 * APART, ws_bytes=1 << 39):
    return lib.gsz_relpos_bias_grad(dy, dt, buckets, heads, far, both, batch, q, k, start, starts, st, scale, g, gt, acc, ws, ws_bytes, None)


BIG = dict(rows=200, cols=300)           # matrices that need a workspace
MANY = dict(BIG, numel=(60000, 5, 60000))
SIZES = [(dict(heads=-1), INVALID), (dict(batch=-1), INVALID), (dict(q=-1), INVALID), (dict(k=-1), INVALID), (dict(heads=1 << 17), SIZE),
         (dict(batch=(1 << 30) + 1), SIZE), (dict(q=(1 << 30) + 1), SIZE), (dict(k=(1 << 30) + 1), SIZE),
         (dict(batch=1 << 20, q=1 << 20, k=1 << 20), SIZE), (dict(buckets=1), INVALID), (dict(buckets=257), INVALID), (dict(buckets=3), INVALID),
         (dict(buckets=2), INVALID), (dict(buckets=33), INVALID), (dict(far=8), INVALID), (dict(far=16, both=0), INVALID),
         (dict(far=(1 << 30) + 1), INVALID), (dict(both=2), INVALID), (dict(start=(1 << 40) + 1), INVALID), (dict(starts=BUF, st=BF16), INVALID),
         (dict(starts=BUF + 4), MISALIGNED), (dict(starts=BUF + 2, st=I32), MISALIGNED), (dict(scale=NAN), INVALID), (dict(scale=1e39), INVALID)]


@pytest.mark.parametrize("call,kw,want", [
    (orth, dict(t=2), INVALID), (orth, dict(count=-1), INVALID), (orth, dict(rows=-1), INVALID), (orth, dict(cols=-1), INVALID),
    (orth, dict(rows=(1 << 17) + 1), SIZE), (orth, dict(cols=(1 << 17) + 1), SIZE), (orth, dict(rows=1 << 17, cols=(1 << 15) + 1), SIZE),
    (orth, dict(count=(1 << 31) + 1), SIZE), (orth, dict(count=1 << 31, rows=1 << 10, cols=1 << 10), SIZE), (orth, dict(steps=0), INVALID), (orth, dict(steps=17), INVALID), (orth, dict(eps=0.0), INVALID),
    (orth, dict(eps=-1.0), INVALID), (orth, dict(eps=NAN), INVALID), (orth, dict(eps=INF), INVALID), (orth, dict(steps=1, ns=[1.0, NAN, 0.0]), INVALID),
    (orth, dict(steps=1, ns=[1.0, 0.0, 1e5]), INVALID), (orth, dict(x=None), INVALID), (orth, dict(out=None), INVALID),
    (orth, dict(x=BUF + 1), MISALIGNED), (orth, dict(t=F32, x=BUF + 2), MISALIGNED), (orth, dict(out=APART + 1), MISALIGNED),
    (orth, dict(BIG, ws=None), SIZE), (orth, dict(BIG, ws_bytes=16), SIZE), (orth, dict(BIG, ws=2 * APART + 8), MISALIGNED),
    (orth, dict(rows=129, cols=129, ws=None), SIZE), (orth, dict(rows=257, cols=2, ws=None), SIZE),
    (orth, dict(out=BUF + 2), INVALID), (orth, dict(t=F32, out=BUF), INVALID), (orth, dict(BIG, ws=BUF), INVALID), (orth, dict(BIG, ws=APART), INVALID),
    (muon, dict(no_plan=True), INVALID), (muon, dict(no_hp=True), INVALID), (muon, dict(no_list=True), INVALID), (muon, dict(count=-1), INVALID),
    (muon, dict(tensors=(0, 3)), INVALID), (muon, dict(tensors=(-1,)), INVALID), (muon, dict(tensors=(2, 0, 2)), INVALID),
    (muon, dict(tensors=(0, 1)), SIZE), (muon, dict(rows=8, cols=8), SIZE), (muon, dict(nesterov=False, steps=0), INVALID),
    (muon, dict(lr=NAN), INVALID), (muon, dict(lr=INF), INVALID), (muon, dict(momentum=NAN), INVALID), (muon, dict(weight_decay=INF), INVALID),
    (muon, dict(scale=1e300), INVALID), (muon, dict(eps=0.0), INVALID),
    (muon, dict(w=None), INVALID), (muon, dict(m=None), INVALID), (muon, dict(g=None), INVALID), (muon, dict(coef=None), INVALID), (muon, dict(p=None), INVALID),
    (muon, dict(w=BUF + 8), MISALIGNED), (muon, dict(m=APART + 4), MISALIGNED), (muon, dict(g=APART + 4), MISALIGNED), (muon, dict(p=APART + 2), MISALIGNED),
    (muon, dict(coef=BUF + 2), MISALIGNED), (muon, dict(MANY, ws=None), SIZE), (muon, dict(MANY, ws_bytes=64), SIZE), (muon, dict(MANY, ws=BUF + 8), MISALIGNED),
    (muon, dict(m=BUF), INVALID), (muon, dict(g=BUF), INVALID), (muon, dict(g=APART), INVALID), (muon, dict(p=BUF + 64), INVALID), (muon, dict(MANY, ws=BUF), INVALID),
    (muon, dict(coef=BUF + 4), INVALID),
    (bias, dict(tt=2), INVALID), (bias, dict(ot=-1), INVALID), (bias, dict(table=None), INVALID), (bias, dict(out=None), INVALID),
    (bias, dict(table=BUF + 1), MISALIGNED), (bias, dict(ot=F32, out=APART + 2), MISALIGNED), (bias, dict(add=BUF + 1), MISALIGNED),
    (bias, dict(out=BUF), INVALID), (bias, dict(add=APART + 2), INVALID), (bias, dict(starts=APART), INVALID),
    (grad, dict(dt=3), INVALID), (grad, dict(gt=2), INVALID), (grad, dict(acc=2), INVALID), (grad, dict(dy=None), INVALID), (grad, dict(g=None), INVALID),
    (grad, dict(dy=BUF + 1), MISALIGNED), (grad, dict(g=APART + 2), MISALIGNED), (grad, dict(ws=None), SIZE), (grad, dict(ws_bytes=8), SIZE),
    (grad, dict(ws=2 * APART + 8), MISALIGNED), (grad, dict(g=BUF), INVALID), (grad, dict(ws=BUF), INVALID), (grad, dict(ws=APART), INVALID),
    (grad, dict(starts=APART), INVALID), (grad, dict(starts=2 * APART), INVALID),
] + [(c, kw, want) for c in (bias, grad) for kw, want in SIZES])
def test_refusals(call, kw, want):
    lib = G.load()
    assert call(lib, **kw) == want, (lib.gsz_last_error(), kw)
    assert lib.gsz_last_error().startswith((b"gsz_orthogonalize", b"gsz_muon", b"gsz_relpos"))


def test_workspace_bytes():
    up = lambda v, m: (v + m - 1) // m * m  # noqa: E731
    for count, rows, cols in ((1, 1, 257), (3, 700, 9), (24, 2048, 2048), (300, 16, 400), (1, 28672, 8192), (40, 129, 129), (256, 100, 5000)):
        b = G.muon_workspace_bytes(count, rows, cols)
        n, small, large = min(count, 256), min(rows, cols), max(rows, cols)
        least = 2 * n * up(small, 32) * up(large, 128) if small <= 128 else 4 * n * (up(rows, 64) * up(cols, 64) + up(small, 64) ** 2)
        assert b % 256 == 0 and least <= b
        assert b <= least + (4 * n * 128 * 128 if small <= 128 else 2 * n * up(small, 64) ** 2) + (64 << 20) + 8 * n * (rows * cols // 4096 + 2) + 2048
        assert b >= G.muon_workspace_bytes(count - 1, rows, cols)
    for rows, cols in ((1, 1), (128, 256), (256, 128), (128, 128)):
        assert G.muon_workspace_bytes(300, rows, cols) == 0
    assert G.muon_workspace_bytes(0, 5, 5) == G.muon_workspace_bytes(5, 0, 5) == 0
    assert G.relpos_bias_workspace_bytes(0, 2, 3, 4, 32) == 0
    for args in ((1, 1, 1, 1, 2), (8, 12, 1024, 1024, 32), (2, 32, 4096, 4096, 256)):
        b = G.relpos_bias_workspace_bytes(*args)
        batch, heads, q, k, buckets = args
        assert 4 * heads * buckets * batch <= b <= 4 * heads * buckets * batch * -(-q // 16) * (2 + (k + 255) // 1024)
    for bad in ((-1, 1, 1), (1, -1, 1), (1, 1, (1 << 17) + 1)):
        with pytest.raises(G.GszError):
            G.muon_workspace_bytes(*bad)
    for bad in ((1, 1, 1, 1, 1), (-1, 1, 1, 1, 2)):
        with pytest.raises(G.GszError):
            G.relpos_bias_workspace_bytes(*bad)
    assert G.load().gsz_muon_workspace_bytes(1, 1, 1, None) == INVALID
    assert G.load().gsz_relpos_bias_workspace_bytes(1, 1, 1, 1, 2, None) == INVALID


def test_binding_refusals():
    import torch
    bf, f32, i64 = torch.bfloat16, torch.float32, torch.int64
    x, out = Dev((2, 6, 8), f32), Dev((2, 6, 8), bf)
    for args, match in (((x, Dev((2, 6, 9), bf)), "out has 108"), ((x, x), "out has dtype"), ((Dev((6,), f32), out), "2-D or 3-D"),
                        ((Dev((2, 6, 8), torch.float16), out), "x has dtype"), ((None, out), "2-D or 3-D")):
        with pytest.raises(ValueError, match=match):
            G.orthogonalize(*args, None, stream=0)
    with pytest.raises(ValueError, match="ns holds 4"):
        G.orthogonalize(x, out, None, steps=5, ns=[(1.0, 0.0, 0.0)] * 4, stream=0)
    with pytest.raises(ValueError, match="ns holds 2"):
        G.make_muon_hp(0.1, steps=2, ns=[(1.0, 0.0)] * 2)
    with pytest.raises(ValueError, match="device tensor"):
        G.orthogonalize(torch.zeros(2, 3), torch.zeros(2, 3, dtype=bf), None, stream=0)
    plan, hp = G.Plan([48, 48], 1 << 20, 2), G.make_muon_hp(0.1)
    n = plan.flat_len
    good = dict(master=Dev((n,), f32), momentum=Dev((n,), f32), g=Dev((n,), f32), coef=Dev((1,), f32), params=Dev((n,), bf))
    for name, bad, match in (("master", Dev((n,), bf), "master has dtype"), ("momentum", Dev((n,), bf), "momentum has dtype"),
                             ("g", Dev((n - 1,), f32), "g has"), ("params", Dev((n,), f32), "params has dtype"), ("params", Dev((n - 1,), bf), "params has"),
                             ("coef", Dev((0,), f32), "coef has"), ("master", Dev((n - 1,), f32), "master has")):
        kw = dict(good, **{name: bad})
        with pytest.raises(ValueError, match=match):
            G.muon_step(plan, [0], 6, 8, kw["master"], kw["momentum"], kw["g"], kw["coef"], hp, kw["params"], None, stream=0)
    with pytest.raises(ValueError, match="master is required"):
        G.muon_step(plan, [0], 6, 8, None, good["momentum"], good["g"], good["coef"], hp, good["params"], None, stream=0)
    with pytest.raises(ValueError, match="make_muon_hp"):
        G.muon_step(plan, [0], 6, 8, *(good[k] for k in ("master", "momentum", "g", "coef")), G.make_hp(0.1, 0.9, 0.9, 1e-8, 0.1, 1), good["params"], None, stream=0)
    # coefficients of fewer steps than the call would read
    longer = G.make_muon_hp(0.1, steps=2, ns=[(1.5, -0.5, 0.0)] * 2)
    longer.steps = 5
    with pytest.raises(ValueError, match="was changed"):
        G.muon_step(plan, [0], 6, 8, *(good[k] for k in ("master", "momentum", "g", "coef")), longer, good["params"], None, stream=0)
    table, s = Dev((32, 2), bf), Dev((1, 2, 3, 4), bf)
    for args, kw, match in (((Dev((64,), bf), s), {}, "2-D"), ((table, Dev((2, 3, 4), bf)), {}, "4-D"), ((table, Dev((1, 3, 3, 4), bf)), {}, "3 heads"),
                            ((table, s), dict(add=Dev((1, 2, 3, 4), f32)), "add has dtype"), ((table, s), dict(add=Dev((1, 2, 3, 5), bf)), "add has 30"),
                            ((table, s), dict(q_start=Dev((2,), i64)), "q_start has 2"), ((table, s), dict(q_start=Dev((1,), f32)), "q_start has dtype"),
                            ((table, Dev((1, 2, 3, 4), torch.float16)), {}, "out has dtype")):
        with pytest.raises(ValueError, match=match):
            G.relpos_bias(*args, 128, stream=0, **kw)
        if "add" not in kw:
            with pytest.raises(ValueError, match=match.replace("out", "dy")):
                G.relpos_bias_grad(args[1], args[0], None, 128, stream=0, **kw)


def test_they_neither_allocate_nor_wait():
    banned = re.compile(r"\b(hipMalloc\w*|hipFree\w*|hipExtMalloc\w*|hipHostMalloc|hipDeviceSynchronize|"
                        r"hipStreamSynchronize|hipEventSynchronize|hipMemcpy\w*|hipMemset\w*)\s*\(")
    for folder in ("optim", "matrix"):
        path = os.path.join(os.path.dirname(G.LIB_PATH), folder)
        for name in sorted(os.listdir(path)):
            assert not banned.search(open(os.path.join(path, name)).read()), name
