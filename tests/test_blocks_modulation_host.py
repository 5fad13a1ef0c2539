"""Rows of a modulation for a run of residual blocks, without a GPU."""

import pytest
import torch

from block_sparse_attention_sparge_gb300 import train as T
from test_blocks_host import Crossing, Plain, _join


@pytest.mark.parametrize("rows", [1, 3, 4])
def test_one_row_for_each_block_that_takes_one(monkeypatch, rows):
    """Two of three blocks take a row each. One for every block of the stack would give the
    second its neighbour's row without a word."""
    monkeypatch.setattr(T, "residual_norm", _join)
    blocks = [Plain(), Crossing(), Plain()]
    x, context = torch.ones(1, 4, 8), torch.zeros(1, 2, 8)
    with pytest.raises(ValueError, match="2 blocks"):
        T.run_blocks(blocks, x, modulation=torch.ones(1, 1, rows, 3, 8), context=context)
    T.run_blocks(blocks, x, modulation=torch.ones(1, 1, 2, 3, 8), context=context)


def test_blocks_that_all_cross(monkeypatch):
    monkeypatch.setattr(T, "residual_norm", _join)
    x, context = torch.ones(1, 4, 8), torch.zeros(1, 2, 8)
    with pytest.raises(ValueError):
        T.run_blocks([Crossing()], x, modulation=torch.ones(1, 1, 1, 3, 8), context=context)
    T.run_blocks([Crossing()], x, context=context)


def test_self_attention_alone_takes_its_first_rows_as_before(monkeypatch):
    monkeypatch.setattr(T, "residual_norm", _join)
    x = torch.ones(1, 4, 8)
    y = T.run_blocks([Plain()], x, modulation=torch.ones(1, 1, 2, 3, 8))
    assert torch.equal(y, x * 3)
