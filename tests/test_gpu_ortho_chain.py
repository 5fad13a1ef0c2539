"""Steps on rows that begin anywhere: a momentum's neighbours in one 32-byte piece are written by
other CTAs of the kernel before the one that reads them all."""

import pytest
import torch

from block_sparse_attention_sparge_gb300 import binding as B
from ortho_reference import ROUND, reference

pytestmark = pytest.mark.gpu


def _rand(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).cuda()


@pytest.mark.parametrize("shape", [(300, 1001), (1001, 300), (64, 2049), (700, 129), (1290, 1027)])
def test_momenta_are_the_new_ones(shape):
    """The gradient outweighs the momentum, so an old value in the new one's place is off by
    more than its own size; every step is repeated bit for bit from the same state."""
    w = torch.zeros(shape, device="cuda")
    m = _rand(1, *shape)
    for step in range(30):
        g = 10 * _rand(2 + step, *shape)
        again = w.clone(), m.clone()
        want_m = 0.9 * m.double() + g.double()
        w0 = w.double()
        B.sparge_muon_step([w], [g], [m], 0.1, momentum=0.9, rms=1.0)
        B.sparge_muon_step([again[0]], [g], [again[1]], 0.1, momentum=0.9, rms=1.0)
        assert torch.equal(again[0], w) and torch.equal(again[1], m)
        # (mu as fp32, one product and one sum)
        off = 3 * 2.0 ** -24 * ((want_m - g.double()).abs() + g.double().abs())
        assert ((m.double() - want_m).abs() <= off).all()
        o = 0.1 * max(shape) ** 0.5 * reference(g.double() + 0.9 * want_m)
        want = w0 - o
        # (the exact form's 2^-17 of the step; the weight's rounding and the step's, as fp32)
        assert (w.double() - want).norm() <= 2.0 ** -17 * o.norm() + 2 * ROUND[w.dtype] * (
            want.norm() + o.norm())
        # single values: an error spread evenly stays below some six of its rms
        assert (w.double() - want).abs().max() <= 24 * 2.0 ** -17 * max(
            o.abs().max(), want.abs().max())
