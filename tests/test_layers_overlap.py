"""Buffers that a layer call writes over what it reads are refused before any device
call; neighbours that touch, and dropout in place, are not among them."""
import pytest

import gradient_sync_zero_amd as G
from tests.test_layers_cpu import F32, I32, INVALID, drop, grad, lookup

A, FAR = 1 << 30, 1 << 40        # addresses that no refused call reads


@pytest.mark.parametrize("call,kw", [
    # 16 values: y one value into x or add, before or after; over the random state
    (drop, dict(x=A, y=A + 2)), (drop, dict(x=A + 30, y=A)), (drop, dict(x=FAR, y=A, add=A + 2)),
    (drop, dict(x=A, y=A, add=A + 30)), (drop, dict(x=A, y=A + 60, t=F32)),
    (drop, dict(x=A, y=A + 32, add=A + 32 + 2)), (drop, dict(x=FAR, y=A, rng=A + 24)), (drop, dict(x=FAR, y=A, rng=A - 8)),
    # 10 rows of 8 and 4 tokens: out is 64 bytes, the table 160, the ids 32
    (lookup, dict(table=FAR, ids=A, out=A)), (lookup, dict(table=FAR, ids=A, out=A + 30)),
    (lookup, dict(table=FAR, ids=A + 56, out=A)), (lookup, dict(table=A, ids=FAR, out=A + 158)),
    (lookup, dict(table=A + 62, ids=FAR, out=A)), (lookup, dict(table=A, ids=FAR, out=A, tt=F32, ot=F32)),
    (lookup, dict(table=FAR, ids=FAR * 2, out=A, p=0.5, rng=A + 56)),
    (grad, dict(ids=FAR, dy=A, g=A)), (grad, dict(ids=FAR, dy=A + 158, g=A)), (grad, dict(ids=FAR, dy=A, g=A + 62)),
    (grad, dict(ids=A + 152, dy=FAR, g=A)), (grad, dict(ids=A, it=I32, dy=FAR, g=A + 14, acc=1)),
    (grad, dict(ids=FAR, dy=FAR * 2, g=A, p=0.5, rng=A + 152)),
    # 200 tokens: a workspace over the gradient, over dy, over the ids
    (grad, dict(n=200, ids=FAR, dy=FAR * 2, g=A, ws=A)), (grad, dict(n=200, ids=FAR, dy=FAR * 2, g=A, ws=A + 144)),
    (grad, dict(n=200, ids=FAR, dy=A, g=FAR * 2, ws=A + 3184)), (grad, dict(n=200, ids=A, dy=FAR, g=FAR * 2, ws=A - 256)),
])
def test_refused(call, kw):
    lib = G.load()
    assert call(lib, **kw) == INVALID, (lib.gsz_last_error(), kw)
    assert b"overlap" in lib.gsz_last_error()
