"""Forms of the embedding and dropout calls beside those of test_gpu_embedding:
one workspace for batches of every size.  Bounds as there."""
import numpy as np
import pytest
import torch

import gradient_sync_zero_amd as G
from oracle import embedding as E
from tests.test_gpu_embedding import BF, EPS, F32, SEED, SITE, STEP, U, draw, f64, make_ids, near, out_bound, rng_tensor

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("most,dim", [(8192, 1024), (20_000, 40)])
def test_one_workspace_for_every_batch(most, dim):
    """A workspace of the largest batch's bytes, and no more, serves the smaller ones."""
    rows = 300
    rng = np.random.default_rng(most)
    ws = torch.empty(G.embedding_workspace_bytes(most, rows, dim), dtype=torch.uint8, device="cuda")
    for n in (most, most - 32, most // 2 + 1, most // 4, 1000, 129, 128, 1, 0):
        ids = torch.from_numpy(make_ids("hot", n, rows, rng)).cuda()
        dy = draw(rng, (n, dim), BF)
        grad = torch.full((rows, dim), float("nan"), device="cuda")
        G.embedding_grad(ids, dy, grad, ws, scale=2.0)
        i = ids.cpu().numpy()
        ref, size = E.grad(i, f64(dy), rows, 2.0)
        m = np.bincount(i, minlength=rows).astype(float)[:, None]
        near(grad, ref, size * ((1 + EPS) ** (m + 3) - 1) * (1 + EPS) ** 2 + out_bound(ref, F32, 1), (n, dim))


@pytest.mark.parametrize("n", [4, 700, 9000])
def test_a_table_of_as_many_rows_as_there_may_be(n):
    """2^31 - 1 rows of one column, written whole: more rows than the launches that
    clear have blocks for.  Small whole numbers, so the sums are exact."""
    rows = (1 << 31) - 1
    rng = np.random.default_rng(n)
    at = np.unique(np.concatenate([rng.integers(0, rows, n), [0, 1, rows - 2, rows - 1]]))[-n:]
    ids = torch.from_numpy(np.resize(at, n)).cuda()
    dy = torch.from_numpy(rng.integers(1, 9, n).astype(np.float32)).to(BF).cuda().view(n, 1)
    grad = torch.full((rows, 1), 3.0, dtype=BF, device="cuda")
    ws = torch.empty(G.embedding_workspace_bytes(n, rows, 1), dtype=torch.uint8, device="cuda")
    G.embedding_grad(ids, dy, grad, ws)
    want = np.zeros(at.size)
    np.add.at(want, np.arange(n) % at.size, f64(dy)[:, 0])
    assert np.array_equal(f64(grad[torch.from_numpy(at).cuda(), 0]), want)
    assert int((grad != 0).sum()) == at.size
    del grad, ws
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_dropout_past_32_bits(dtype):
    """2^32 + 5003 elements: places on both sides of 2^32 keep and drop what the
    generator says and hold the kept values exactly doubled."""
    n = (1 << 32) + 5003
    x = torch.full((n,), 1.5, dtype=dtype, device="cuda")
    x[-5003:] = torch.arange(1, 5004, device="cuda").remainder(64).add(1).to(dtype)
    G.dropout(x, x, 0.5, rng_tensor(), SITE)
    for first, m in ((0, 4099), ((1 << 31) - 2000, 4000), ((1 << 32) - 3000, 8003)):
        kept = E.kept(first, m, 0.5, SEED, STEP, SITE)
        e = np.arange(first, first + m)
        was = np.where(e < 1 << 32, 1.5, (e - (1 << 32) + 1) % 64 + 1.0)
        assert 0.4 < kept.mean() < 0.6
        assert np.array_equal(f64(x[first:first + m]), np.where(kept, 2 * was, 0.0)), first
    del x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("p", [0.0, 0.5])
@pytest.mark.parametrize("dim", [65_544, 65_541])
def test_lookup_past_32_bits(dim, p):
    """Rows of the table and of out on both sides of element 2^32, all of them full of
    values, against the oracle's mask and an exact doubling."""
    n, rows = 65_600, 65_700
    ids = (torch.arange(n, device="cuda") * 7919) % rows
    table = torch.empty(rows, dim, dtype=BF, device="cuda")
    table.copy_(torch.arange(rows, device="cuda").remainder(61).add(1)[:, None].expand(rows, dim))
    table += torch.arange(dim, device="cuda").remainder(2).to(BF)          # odd columns one more
    out = torch.full((n, dim), float("nan"), dtype=BF, device="cuda")
    G.embedding_lookup(ids, table, out, scale=2.0, p=p, rng=rng_tensor(), site=SITE)
    k = 2.0 * E.keep_scale(p)
    border = (1 << 32) // dim
    far = int((ids > border).nonzero()[0, 0])
    for i in (0, 1, far, border - 1, border, border + 1, n - 1):
        kept = E.kept(i * dim, dim, p, SEED, STEP, SITE)
        want = np.where(kept, (int(ids[i]) % 61 + 1 + np.arange(dim) % 2) * k, 0.0)
        assert want.any() and np.array_equal(f64(out[i]), want), (i, int(ids[i]))
    assert bool(torch.isfinite(out).all())
    del table, out
    torch.cuda.empty_cache()


# A lane takes two vectors of 8 columns from 2^21 vectors in the call on, four from 2^22
# on; rows lie side by side in a block up to 128 vectors, and longer ones are cut into
# pieces of at most 256.
@pytest.mark.parametrize("n,dim", [(2_200_003, 1), (4_200_003, 1), (1_100_003, 9), (300_007, 100), (33_001, 1016), (33_001, 1030),
                                   (17_001, 2060), (11_003, 2048), (5601, 6150), (2207, 8200), (4241, 8193)])
@pytest.mark.parametrize("tt,ot,it", [(BF, BF, torch.int64), (F32, BF, torch.int32), (BF, F32, torch.int32), (F32, F32, torch.int64)])
def test_lookup_of_several_vectors_a_lane(n, dim, tt, ot, it):
    """Every value of large lookups, from and to odd places, against the table's rows
    doubled (exact in each type)."""
    assert n * (-(-dim // 8)) >= 1 << 21
    rows, shift = 1009, 3
    gen = torch.Generator(device="cuda").manual_seed(n)
    tbuf = torch.randn(rows * dim + shift, device="cuda", generator=gen).to(BF).to(tt)
    table = tbuf[shift:].view(rows, dim)
    ids = torch.randint(-3, rows + 3, (n,), device="cuda", generator=gen).to(it)
    obuf = torch.full((n * dim + shift + 8,), float("nan"), dtype=ot, device="cuda")
    obuf[:shift], obuf[shift + n * dim:] = 7.25, 7.25
    out = obuf[shift:shift + n * dim].view(n, dim)
    G.embedding_lookup(ids, table, out, scale=2.0)
    ok = (ids >= 0) & (ids < rows)
    want = (table * 2).to(ot).index_select(0, ids.clamp(0, rows - 1).long())
    want[~ok] = 0
    assert torch.equal(out, want)
    assert bool((obuf[:shift] == 7.25).all()) and bool((obuf[shift + n * dim:] == 7.25).all()), "wrote outside"


@pytest.mark.parametrize("rows", [(1 << 19) - 1, 1 << 19, 600_001])
@pytest.mark.parametrize("n", [129, 700, 8191, 8192])
@pytest.mark.parametrize("acc,kind", [(False, "any"), (True, "any"), (False, "hot"), (True, "ends")])
def test_grad_of_some_tokens_on_tall_tables(rows, n, acc, kind):
    """The compare-all sort where a row's number and a token's position just fit, or do
    not fit, one 32-bit key."""
    dim = 3
    rng = np.random.default_rng(rows + n)
    i = np.where(rng.random(n) < 0.5, rows - 1, rng.choice([0, rows - 2, rows, -1], n)) if kind == "ends" else make_ids(kind, n, rows, rng)
    i[:2] = rows - 1, rows
    ids, dy = torch.from_numpy(i).cuda(), draw(rng, (n, dim), F32)
    old = draw(rng, (rows, dim), F32)
    grad = old.clone() if acc else torch.full_like(old, float("nan"))
    ws = torch.full((G.embedding_workspace_bytes(n, rows, dim) // 4,), float("nan"), device="cuda")
    G.embedding_grad(ids, dy, grad, ws, scale=0.5, accumulate=acc)
    ref, size = E.grad(i, f64(dy), rows, 0.5, old=f64(old) if acc else None)
    m = np.bincount(i[(i >= 0) & (i < rows)], minlength=rows).astype(float)[:, None]
    near(grad, ref, size * ((1 + EPS) ** (m + 3) - 1) * (1 + EPS) ** 2 + out_bound(ref, F32, 1), (rows, n, kind))
    rest = torch.from_numpy(m[:, 0] == 0).cuda()
    assert torch.equal(grad[rest], old[rest] if acc else torch.zeros_like(old[rest]))


def test_grad_of_as_many_tokens_as_there_may_be():
    """2^30 tokens (the sort's tiles go over 8192 rounds each), small whole numbers, about
    1074 tokens a row: every sum is exact in fp32."""
    n, rows = 1 << 30, 1_000_003
    ids = torch.arange(n, dtype=torch.int32, device="cuda").remainder_(rows)
    dy = torch.arange(n, dtype=torch.int32, device="cuda").bitwise_right_shift_(7).remainder_(5).to(BF).view(n, 1)
    grad = torch.full((rows, 1), float("nan"), device="cuda")
    ws = torch.empty(G.embedding_workspace_bytes(n, rows, 1), dtype=torch.uint8, device="cuda")
    G.embedding_grad(ids, dy, grad, ws)
    want = torch.zeros(rows, dtype=torch.float64, device="cuda")
    for a in range(0, n, 1 << 27):
        want.index_add_(0, ids[a:a + (1 << 27)].long(), dy[a:a + (1 << 27), 0].double())
    assert float(want.max()) < 1 << 24 and torch.equal(grad[:, 0].double(), want)
    del ids, dy, ws, want
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dim", [1 << 29, (1 << 29) - 3])
def test_rows_as_wide_as_they_may_be(dim):
    """2^29 columns and three fewer: lookup, and the gradient of its three tokens."""
    table = torch.empty(2, dim, dtype=BF, device="cuda")
    for r in range(2):
        table[r] = torch.arange(dim, dtype=torch.int32, device="cuda").remainder_(251 - r).to(BF)
    ids = torch.tensor([1, 2, 1], device="cuda")
    out = torch.full((3, dim), float("nan"), dtype=BF, device="cuda")
    G.embedding_lookup(ids, table, out, scale=2.0)
    assert torch.equal(out[0], table[1] * 2) and torch.equal(out[2], out[0]) and not bool(out[1].any())
    out[1] = 9.0
    grad = torch.full((2, dim), float("nan"), dtype=BF, device="cuda")
    G.embedding_grad(ids, out, grad, None, scale=0.25)
    assert torch.equal(grad[1], table[1]) and not bool(grad[0].any())
    del table, out, grad
    torch.cuda.empty_cache()


@pytest.mark.parametrize("bucket", [BF, F32])
def test_beside_the_calls_that_pack_every_tensor(bucket):
    """The table's gradient in a bucket that bucket_pack and bucket_accumulate fill: those
    write every tensor's place, so they go first, the table's place taking anything when
    packed and zeros when accumulated."""
    rows, dim, n = 300, 101, 500
    rng = np.random.default_rng(9)
    plan = G.Plan([rows * dim, 37, 5000], 1 << 16, 2).upload()
    flat = torch.full((plan.flat_len,), float("nan"), dtype=bucket, device="cuda")
    pack, add = (G.bucket_pack, G.bucket_accumulate) if bucket == BF else (G.bucket_pack_f32, G.bucket_accumulate_f32)
    slot = plan.view(0, flat).view(rows, dim)
    ws = torch.empty(G.embedding_workspace_bytes(n, rows, dim), dtype=torch.uint8, device="cuda")
    total, others = None, [np.zeros(37), np.zeros(5000)]
    for k in range(3):
        fill = torch.zeros(rows * dim, dtype=BF, device="cuda") if k else draw(rng, rows * dim, BF)
        rest = [torch.from_numpy(rng.integers(-8, 9, m).astype(np.float32)).to(BF).cuda() for m in (37, 5000)]
        (add if k else pack)(plan, [fill, *rest], flat)
        i = make_ids("any", n, rows, rng)
        dy = torch.from_numpy(rng.integers(-2, 3, (n, dim)).astype(np.float32)).to(BF).cuda()
        G.embedding_grad(torch.from_numpy(i).cuda(), dy, slot, ws, accumulate=k > 0)
        total = E.grad(i, f64(dy), rows, old=total)[0]
        others = [o + f64(r) for o, r in zip(others, rest)]
    assert np.abs(total).max() <= 256                    # whole numbers that bf16 holds too
    assert np.array_equal(f64(slot), total)
    assert all(np.array_equal(f64(plan.view(t + 1, flat)), o) for t, o in enumerate(others))
    assert bool(torch.isfinite(flat).all())              # the pads are zero
