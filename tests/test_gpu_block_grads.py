"""Gradients as autograd hands them over: contiguous views that begin at any
element of a larger buffer (the pieces of a concatenation's gradient)."""

import pytest
import torch

from block_sparse_attention_sparge_gb300 import binding as B
from block_sparse_attention_sparge_gb300 import train

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def _rand(seed, *shape, dtype=F32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DEV, dtype)


def _grads(outs, weights, leaves, lead):
    """Gradients of sum(outs * weights), the outputs read through a
    concatenation behind ``lead`` other elements."""
    dtype = outs[0].dtype
    flat = torch.cat([torch.zeros(lead, dtype=dtype, device=DEV)] + [o.flatten() for o in outs])
    w = torch.cat([torch.zeros(lead, dtype=dtype, device=DEV)] + [t.flatten() for t in weights])
    return torch.autograd.grad(flat, leaves, w)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_residual_norm(dtype):
    x, br = (_rand(i, 2, 7, 64, dtype=dtype).requires_grad_(True) for i in range(2))
    wy, wh = _rand(3, 2, 7, 64, dtype=dtype), _rand(4, 2, 7, 64, dtype=dtype)
    want = _grads(train.residual_norm(x, br), (wy, wh), (x, br), 0)
    for lead in (1, 3):
        got = _grads(train.residual_norm(x, br), (wy, wh), (x, br), lead)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_qkv_heads():
    leaves = [_rand(i, 1, 9, 2, 64).requires_grad_(True) for i in range(3)]
    weights = [_rand(5 + i, 1, 2, 9, 64, dtype=BF) for i in range(3)]
    want = _grads(train.qkv_heads(*leaves, norm="token"), weights, leaves, 0)
    for lead in (1, 5):
        got = _grads(train.qkv_heads(*leaves, norm="token"), weights, leaves, lead)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_sparse_attention():
    leaves = [_rand(i, 1, 1, 200, 64, dtype=BF).requires_grad_(True) for i in range(3)]
    w = [_rand(5, 1, 1, 200, 64, dtype=BF)]
    want = _grads([train.sparse_attention(*leaves, 0.5, 0.5)], w, leaves, 0)
    got = _grads([train.sparse_attention(*leaves, 0.5, 0.5)], w, leaves, 3)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_the_binding_itself_still_refuses_such_a_gradient():
    x = _rand(1, 7, 64)
    dy = _rand(2, 7 * 64 + 1)[1:].view(7, 64)
    with pytest.raises(B.SpargeError) as e:
        B.sparge_resnorm_bwd(dy, None, x, x.clone(), norm=None)
    assert e.value.code == B.SPARGE_ERR_MISALIGNED
