"""Outputs that the caller gives to sparge_heads_fwd and sparge_heads_bwd: what
autograd is told of them, and where they may lie."""

import pytest
import torch

from block_sparse_attention_sparge_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def _rand(seed, *shape, dtype=BF):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DEV, dtype)


def test_autograd_notices_that_an_output_was_written():
    b, n, h, d = 1, 9, 2, 64
    q, k = _rand(1, b, n, h, d), _rand(2, b, n, h, d)
    leaf = torch.ones((), device=DEV, requires_grad=True)
    out, free = _rand(3, b, h, n, d), _rand(4, b, h, n, d)
    kept = (leaf * out).sum()  # keeps out for its backward
    before = free._version
    B.sparge_heads_fwd(q, None, None, out=(out, free, None))
    assert free._version == before  # not written: there is no k
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        kept.backward()

    buf = _rand(5, b, n, 2 * h * d)
    kept = (leaf * buf).sum()
    parts = [t.unflatten(-1, (h, d)) for t in buf.chunk(2, -1)]
    B.sparge_heads_bwd(None, _rand(6, b, h, n, d), None, None, k, out=(None, parts[1], None))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        kept.backward()
    (leaf * buf).sum().backward()  # of what it holds now
    assert leaf.grad.isfinite()
