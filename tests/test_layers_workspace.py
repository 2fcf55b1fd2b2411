"""The gradient's workspace never shrinks as a call's tokens grow: one sized for the
largest batch serves every smaller one, a captured or allocation-free loop's last
micro-batch among them."""
import pytest

import gradient_sync_zero_amd as G


@pytest.mark.parametrize("dim", [1, 8, 511, 513, 768, 2048, 4097, 8192, 70_000, 1 << 21, (1 << 21) + 1])
@pytest.mark.parametrize("rows", [0, 5, 1023, 50257, 1 << 20])
def test_a_workspace_serves_every_smaller_batch(rows, dim):
    """n across the borders at which the layout changes: one to 3000 tokens, both
    sides of every power of two and of every multiple of 256 up to 2^15 (chunks of
    4, 8, 16 and 32 tokens give way to one another there), and the sort's tiles of
    512 tokens by the 256."""
    near = {max(0, (1 << k) + d) for k in range(2, 31) for d in range(-33, 34)}
    near |= {256 * k + d for k in range(1, 129) for d in (-1, 0, 1)}
    near |= {512 * 256 * k + d for k in (1, 2, 3, 4, 8) for d in (-1, 0, 1)}
    last, at = 0, 0
    for n in sorted(near | set(range(3000))):
        b = G.embedding_workspace_bytes(n, rows, dim)
        assert b >= last, (at, last, n, b)
        last, at = b, n


def test_the_largest_batch_is_not_asked_for_more_than_its_partial_rows():
    """8192 tokens of 8192 columns: sorted pairs, and at most 4096 column tiles'
    worth of chunks at two partial rows each (256 chunks' 16.8 MB as laid out, twice
    that for the batches just below)."""
    b = G.embedding_workspace_bytes(8192, 32000, 8192)
    assert b <= 8 * 8192 + 2 * 4 * 8192 * 512 + 4096
