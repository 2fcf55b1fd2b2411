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
