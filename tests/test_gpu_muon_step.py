"""A training step with both optimizers, as a model with a relative position bias has it: the bias
read in place in the gathered parameters and added to scores, its gradient accumulated over two
micro-batches in place in each rank's fp32 bucket, the tables' plan reduced to shards and updated by
AdamW, the matrices' plan reduced whole and updated by Muon, one clip coefficient over both, and
the next step's bias read from the new parameters.  The step's older parts bit for bit against their
oracles, the new ones within the bounds of their own tests."""
import numpy as np
import pytest
import torch

import gradient_sync_zero_amd as G
from oracle import muon as OM
from oracle import relpos as OR
from oracle import pack as opack
from oracle.adamw import adamw
from oracle.layout import ag_write
from oracle.plan import make_plan
from oracle.reduce import reduce_mean
from tests.parity import assert_bits, host
from tests.test_gpu_embedding import BF, EPS, F32, U, f64, near, out_bound
from tests.test_gpu_muon import norm

pytestmark = pytest.mark.gpu

P, HEADS, BUCKETS, FAR, Q, K = 2, 5, 32, 128, 60, 75
TABLES = [BUCKETS * HEADS, 37, 1001]                   # the bias comes last in its bucket, at an odd place
ROWS, COLS = 48, 96
MATRICES = [ROWS * COLS, 11, ROWS * COLS]              # 11: a tensor that neither update lists


def test_step():
    rng = np.random.default_rng(5)
    tables, matrices = G.Plan(TABLES, 1 << 20, P).upload(), G.Plan(MATRICES, 1 << 20, P).upload()
    otables, omatrices = make_plan(TABLES, 1 << 20, P), make_plan(MATRICES, 1 << 20, P)
    theta = rng.normal(0, 0.5, tables.flat_len).astype(np.float32)
    gathered = torch.from_numpy(theta).to(BF).cuda()
    assert tables.tensor(0)[0] % 8
    table = tables.view(0, gathered).view(BUCKETS, HEADS)
    flats = []
    for r in range(P):
        flat = torch.zeros(tables.flat_len, device="cuda")
        grads = [torch.from_numpy(rng.normal(0, 1e-3, n).astype(np.float32)).to(BF).cuda() for n in TABLES]
        G.bucket_pack_f32(tables, grads, flat)
        slot = tables.view(0, flat).view(BUCKETS, HEADS)
        for k in range(2):
            scores = torch.from_numpy(rng.normal(size=(2, HEADS, Q, K))).to(BF).cuda()
            x = f64(scores)
            G.relpos_bias(table, scores, FAR, q_start=K - Q, add=scores)
            bias = OR.bias(f64(table), [K - Q] * 2, Q, K, FAR, True)
            near(scores, x + bias, out_bound(x + bias, BF, 1), "scores")
            dy = torch.from_numpy(rng.normal(0, 1e-3, (2, HEADS, Q, K))).to(BF).cuda()
            old = f64(slot).copy()
            ws = torch.empty(G.relpos_bias_workspace_bytes(2, HEADS, Q, K, BUCKETS), dtype=torch.uint8, device="cuda")
            G.relpos_bias_grad(dy, slot, ws, FAR, q_start=K - Q, accumulate=k > 0)
            ref, size = OR.grad(f64(dy), [K - Q] * 2, BUCKETS, FAR, True, 1.0, old if k else None)
            near(slot, ref, size * 296 * EPS + out_bound(ref, F32, 1), "gradient in the bucket")
        for t in (1, 2):
            assert torch.equal(tables.view(t, flat), grads[t].float()), "a neighbour's gradient changed"
        flats.append(flat)

    mflats = [torch.from_numpy(rng.normal(0, 1e-3, matrices.flat_len)).to(BF).cuda() for _ in range(P)]
    S = tables.shard_len
    ws = torch.empty(max(G.workspace_bytes(S), G.workspace_bytes(matrices.shard_len)) // 8, dtype=torch.float64, device="cuda")
    partials = torch.zeros(2 * P, dtype=torch.float64, device="cuda")
    gs = [torch.empty(S, device="cuda") for _ in range(P)]
    for r in range(P):
        G.shard_reduce_mean_f32(tables, r, flats, G.LAYOUT_BUCKET_FLAT, gs[r], partials[r:r + 1], ws)
    mg = torch.empty(matrices.flat_len, device="cuda")
    G.allreduce_mean(matrices, mflats, mg, partials[P:], ws)
    coef = torch.empty(1, device="cuda")
    G.clip_coef(partials, 0.05, coef)
    c = host(coef)[0]
    total = sum((host(g).astype(np.float64) ** 2).sum() for g in gs + [mg])
    assert abs(c * (np.sqrt(total) + 1e-6) / 0.05 - 1) < 1e-6 and c < 1

    new, onew = torch.zeros(tables.flat_len, dtype=BF, device="cuda"), np.zeros(tables.flat_len, dtype=np.uint16)
    hp = G.make_hp(lr=2e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1)
    for r in range(P):
        th = opack.owner_view(otables, theta, r)
        og = reduce_mean([opack.owner_view(otables, host(f), r) for f in flats], r)
        assert_bits(host(gs[r]), og, "reduced gradient")
        state = [torch.from_numpy(th.copy()).cuda()] + [torch.zeros(S, device="cuda") for _ in range(2)]
        G.shard_adamw_step(tables, r, *state, gs[r], coef, hp, new)
        ag_write(otables, r, adamw(th, np.zeros(S, np.float32), np.zeros(S, np.float32), og, c, 2e-4, 0.9, 0.95, 1e-8, 0.1, 1)[3], onew)
    assert_bits(host(new), onew, "tables")

    w0 = rng.normal(0, 0.02, matrices.flat_len).astype(np.float32)
    m0 = rng.normal(0, 1e-3, matrices.flat_len).astype(np.float32)
    w, m = torch.from_numpy(w0.copy()).cuda(), torch.from_numpy(m0.copy()).cuda()
    p = torch.zeros(matrices.flat_len, dtype=BF, device="cuda")
    lr, scale = 2e-3, 0.2 * COLS ** 0.5
    G.muon_step(matrices, [0, 2], ROWS, COLS, w, m, mg, coef, G.make_muon_hp(lr, 0.95, 0.1, scale), p,
                torch.empty(G.muon_workspace_bytes(2, ROWS, COLS), dtype=torch.uint8, device="cuda"))
    for t in (0, 2):
        s = slice(matrices.tensor(t)[0], matrices.tensor(t)[0] + ROWS * COLS)
        shape = lambda v: v[s].reshape(ROWS, COLS)  # noqa: E731
        th1, m1, o = OM.update(shape(w0), shape(m0), shape(host(mg)), c, lr, 0.95, 0.1, scale, True)
        assert np.abs(shape(host(m)) - m1).max() < 1e-8
        u = shape(host(mg)).astype(np.float64) * c + 0.95 * m1
        d = norm(shape(host(w)) - th1)
        assert d <= lr * scale * 2 * OM.rounding_bound(u) + 4 * 2.0 ** -24 * norm(th1), d
        assert np.array_equal(host(p.view(torch.uint16))[s], host(w.bfloat16().view(torch.uint16))[s])
    other = slice(matrices.tensor(1)[0], matrices.tensor(1)[0] + 11)
    assert np.array_equal(host(w)[other], w0[other]) and bool((p[other] == 0).all())

    # the next step reads the new table where it lies
    out = torch.empty(1, HEADS, 3, K, device="cuda")
    G.relpos_bias(tables.view(0, new).view(BUCKETS, HEADS), out, FAR)
    ref = OR.bias(f64(tables.view(0, new).view(BUCKETS, HEADS)), [0], 3, K, FAR, True)
    assert np.array_equal(f64(out), ref)
