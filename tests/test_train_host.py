"""Refusals of the autograd functions that need no GPU."""

import pytest
import torch

from block_sparse_attention_sparge_gb300 import train


def test_calls_without_tensors_or_off_the_device_are_refused():
    q = torch.zeros(1, 8, 2, 64)
    for call in (lambda: train.qkv_heads(), lambda: train.qkv_heads(q),
                 lambda: train.residual_norm(torch.zeros(1, 8, 64)),
                 lambda: train.clip_grad_norm_([q.requires_grad_(True), _with_grad()], 1.0)):
        with pytest.raises(ValueError):
            call()


def _with_grad():
    p = torch.zeros(3, requires_grad=True)
    p.grad = torch.ones(3)
    return p
