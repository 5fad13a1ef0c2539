"""How a run of residual blocks calls its blocks, without a GPU."""

import torch

from block_sparse_attention_sparge_gb300 import train as T


class Plain:
    """A self-attention block of a user's own: attend(x, grid), no other attributes."""
    norm = "rms"

    def attend(self, x, grid=None):
        return 2 * x


class Crossing:
    norm, crosses = "rms", True

    def __init__(self):
        self.seen = []

    def attend(self, x, grid=None, context=None, kv_len=None):
        self.seen.append((context, kv_len))
        return 3 * x


def _join(x, branch=None, gate=None, scale=None, shift=None, norm=None, **_):
    x = x if branch is None else x + branch * (1 if gate is None else gate)
    return x, x * (1 if scale is None else scale)


def test_context_goes_to_the_blocks_that_cross(monkeypatch):
    monkeypatch.setattr(T, "residual_norm", _join)
    cross = Crossing()
    x, context, lens = torch.ones(1, 4, 8), torch.zeros(1, 2, 8), torch.tensor([2])
    y = T.run_blocks([Plain(), cross, Plain()], x, context=context, kv_len=lens)
    assert cross.seen == [(context, lens)]
    assert torch.equal(y, x * 3 * 4 * 3)


def test_modulation_has_rows_for_the_others_alone(monkeypatch):
    calls = []

    def join(x, branch=None, gate=None, scale=None, shift=None, norm=None, **_):
        calls.append(tuple(None if t is None else int(t.flatten()[0]) for t in (gate, scale, shift)))
        return x, x

    monkeypatch.setattr(T, "residual_norm", join)
    rows = torch.arange(6.0).reshape(1, 1, 2, 3, 1).expand(1, 1, 2, 3, 8)  # shift, scale, gate
    T.run_blocks([Plain(), Crossing(), Plain()], torch.ones(1, 4, 8), modulation=rows,
                 context=torch.zeros(1, 2, 8))
    # (gate of the block before, scale and shift of the one after)
    assert calls == [(None, 1, 0), (2, None, None), (None, 4, 3), (5, None, None)]
