"""The embedding operators and the shard step together, as a training step uses
them: parameters looked up in place in the gathered buffer, a residual dropout, the
backward pass into the table's place in each rank's buckets over two micro-batches,
then reduce, clip and AdamW of every owner into the gathered buffer, and a lookup in
that.  The embedding's parts against the 64-bit oracle (bounds as in
test_gpu_embedding), the step bit for bit against the shard step's oracle on the
buckets' own bits."""
import numpy as np
import pytest
import torch

import gradient_sync_zero_amd as G
from oracle import embedding as E
from oracle import pack as opack
from oracle.adamw import adamw
from oracle.layout import ag_write
from oracle.norm import clip_coef, sqnorm_partial, total
from oracle.plan import make_plan
from oracle.reduce import reduce_mean
from tests.parity import assert_bits, host
from tests.test_gpu_embedding import BF, EPS, F32, U, f64, near, out_bound

pytestmark = pytest.mark.gpu

ROWS, DIM, P, MICRO, SCALE, PROB = 300, 101, 2, 2, 10.0, 0.1
NUMEL = [ROWS * DIM, 37, 513]            # the table comes last in its bucket, at element 550


@pytest.mark.parametrize("bucket", [BF, F32])
def test_micro_batches_and_shard_step(bucket):
    rng = np.random.default_rng(77)
    plan = G.Plan(NUMEL, 1 << 20, P).upload()
    oplan = make_plan(NUMEL, 1 << 20, P)
    assert plan.tensor(0)[0] * 2 % 16 != 0
    S, L = plan.shard_len, plan.flat_len
    theta = rng.normal(0, 0.02, L).astype(np.float32)
    gathered = torch.from_numpy(theta).to(BF).cuda()
    table = plan.view(0, gathered).view(ROWS, DIM)
    flats = [torch.zeros(L, dtype=bucket, device="cuda") for _ in range(P)]

    for q in range(P):
        others = [[torch.from_numpy(rng.normal(0, 1e-3, n).astype(np.float32)).to(bucket).cuda()
                   for n in NUMEL[1:]] for _ in range(MICRO)]
        slot = plan.view(0, flats[q]).view(ROWS, DIM)
        want_others = [torch.zeros_like(t) for t in others[0]]
        for k in range(MICRO):
            n = [90, 700][k]
            ids = torch.from_numpy(rng.integers(-1, ROWS + 1, n)).cuda()
            key = torch.tensor([1000 + q, k], dtype=torch.int64, device="cuda")    # a seed for each rank
            args = (1000 + q, k)
            h = torch.empty(n, DIM, dtype=BF, device="cuda")
            G.embedding_lookup(ids, table, h, scale=SCALE, p=PROB, rng=key, site=0)
            ref = E.lookup(ids.cpu().numpy(), f64(table), SCALE, PROB, *args, 0)
            near(h, ref, out_bound(ref, BF), "lookup in the gathered buffer")
            y = torch.empty_like(h)
            G.dropout(h, y, PROB, key, 1, add=h)
            drop = E.dropout(f64(h), PROB, *args, 1)
            near(y, f64(h) + drop, np.abs(drop) * 3 * EPS + out_bound(f64(h) + drop, BF, 1), "residual dropout")
            dy = torch.from_numpy(rng.normal(0, 1e-3, (n, DIM)).astype(np.float32)).to(BF).cuda()
            dh = torch.empty_like(dy)
            G.dropout(dy, dh, PROB, key, 1, add=dy)                  # backward of h + dropout(h)
            old = f64(slot).copy()
            ws = torch.empty(G.embedding_workspace_bytes(n, ROWS, DIM), dtype=torch.uint8, device="cuda")
            G.embedding_grad(ids, dh, slot, ws, scale=SCALE, p=PROB, rng=key, site=0, accumulate=k > 0)
            ref, size = E.grad(ids.cpu().numpy(), f64(dh), ROWS, SCALE, PROB, *args, 0, old if k else None)
            m = np.bincount(np.clip(ids.cpu().numpy(), -1, ROWS) + 1, minlength=ROWS + 2)[1:-1, None]
            bound = size * ((1 + EPS) ** (m + 3) - 1) * (1 + U[bucket]) * (1 + EPS) + out_bound(ref, bucket, 1)
            near(slot, ref, bound, f"rank {q} micro-batch {k}: gradient in the bucket")
            for t, src, acc in zip((1, 2), others[k], want_others):
                plan.view(t, flats[q]).add_(src)
                acc.add_(src)
        used = torch.zeros(L, dtype=torch.bool, device="cuda")
        for t in range(3):
            plan.view(t, used).fill_(True)
            if t:
                assert torch.equal(plan.view(t, flats[q]), want_others[t - 1]), "a neighbour's gradient changed"
        assert bool((flats[q][~used] == 0).all()), "pads"

    # the step on these buckets
    hp = G.make_hp(lr=2e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1)
    ws = torch.empty(G.workspace_bytes(S) // 8, dtype=torch.float64, device="cuda")
    partials = torch.zeros(P, dtype=torch.float64, device="cuda")
    gs = [torch.empty(S, device="cuda") for _ in range(P)]
    reduce = G.shard_reduce_mean if bucket == BF else G.shard_reduce_mean_f32
    for r in range(P):
        reduce(plan, r, flats, G.LAYOUT_BUCKET_FLAT, gs[r], partials[r:r + 1], ws)
    coef = torch.empty(1, device="cuda")
    G.clip_coef(partials, 1.0, coef)
    new = torch.zeros(L, dtype=BF, device="cuda")
    oflats = [host(f) for f in flats]
    og = [reduce_mean([opack.owner_view(oplan, f, r) for f in oflats], r) for r in range(P)]
    _, ocoef = clip_coef(total([sqnorm_partial(g) for g in og]), 1.0)
    onew = np.zeros(L, dtype=np.uint16)
    for r in range(P):
        th = opack.owner_view(oplan, theta, r)
        state = [torch.from_numpy(th.copy()).cuda()] + [torch.zeros(S, device="cuda") for _ in range(2)]
        G.shard_adamw_step(plan, r, *state, gs[r], coef, hp, new)
        p = adamw(th, np.zeros(S, np.float32), np.zeros(S, np.float32), og[r], ocoef, 2e-4, 0.9, 0.95, 1e-8, 0.1, 1)[3]
        ag_write(oplan, r, p, onew)
        assert_bits(host(gs[r]), og[r], f"g of owner {r}")
    torch.cuda.synchronize()
    assert_bits(host(new), onew, "gathered parameters")
    # and the next micro-batch reads them where they lie
    ids = torch.arange(ROWS, device="cuda")
    out = torch.empty(ROWS, DIM, dtype=BF, device="cuda")
    G.embedding_lookup(ids, plan.view(0, new).view(ROWS, DIM), out)
    assert torch.equal(out.view(-1), plan.view(0, new))
    assert not torch.equal(out.view(-1), plan.view(0, gathered))
