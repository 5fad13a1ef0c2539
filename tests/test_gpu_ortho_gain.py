"""The gain of a step: by outputs over inputs, whichever a weight has first."""

import math

import pytest
import torch

from block_sparse_attention_sparge_gb300 import binding as B
from ortho_reference import check, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(60, 200), (200, 60), (130, 130)])
def test_inputs_first(shape):
    gen = torch.Generator().manual_seed(1)
    g = torch.randn(shape, generator=gen).cuda()
    gain = math.sqrt(max(1, shape[1] / shape[0]))
    w = torch.zeros(shape, device="cuda")
    B.sparge_muon_step([w], [g], None, 0.5, inputs_first=True)
    check(w, -0.5 * gain * reference(g), False)
    # the same weight seen as [outputs, inputs]
    t = torch.zeros(shape, device="cuda")
    B.sparge_muon_step([t.t()], [g.t()], None, 0.5)
    assert torch.equal(t, w)
    # a root mean square has no sides
    for kw in (dict(rms=0.2), dict(rms=0.2, inputs_first=True)):
        w.zero_()
        B.sparge_muon_step([w], [g], None, 0.5, **kw)
        check(w, -0.5 * 0.2 * math.sqrt(max(shape)) * reference(g), False)
