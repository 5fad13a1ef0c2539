"""Gradients of the attention over a context whose value rows share a mean, which they do not
depend on: dS = P (dP - D) has differences of values alone.

What the whole gradients may be off by, in the 2-norm. A rounding to bf16 is off by at most HALF
= 2^-8 of the value and evenly spread, so by HALF / sqrt(3) in the mean square at most; roundings
of thousands of values are independent. dQ and dK have two, dS's and the result's: HALF *
sqrt(2 / 3) = 0.0032. Up to 64 keys of capacity D is a sum of P dP in fp32, and that is all.
Beyond, D is taken from O as it was rounded: by row it is off by the sum of dO times O's two
errors, O's own rounding and that of P in the product, Sum_c dO_c^2 (O_c^2 + Sum_j P_j^2 V_jc^2)
* HALF^2 / 3 in the square, which dQ has times P K and dK times P and Q."""

import pytest
import torch

from block_sparse_attention_sparge_gb300 import binding as B
from cross_reference import HALF, reference

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
TWO = HALF * (2 / 3) ** 0.5


def _make(m, d, mean, seed=1, h=2, n=2000):
    g = torch.Generator().manual_seed(seed)
    q, k, v, do = (torch.randn(s, generator=g) for s in
                   ((1, h, n, d), (1, h, m, d), (1, h, m, d), (1, h, n, d)))
    v = v + mean * torch.randn((1, h, 1, d), generator=g)
    return [t.to(BF).cuda() for t in (q, k, v, do)]


def _of_D(q, k, v, do, n):
    """The squares of what O's errors add to dQ and to dK."""
    Q, K, V, G = (t.double() for t in (q, k[:, :, :n], v[:, :, :n], do))
    scale = Q.shape[-1] ** -0.5
    P = (scale * Q @ K.transpose(-1, -2)).softmax(-1)
    square = (G.square() * ((P @ V).square() + P.square() @ V.square())).sum(-1) * HALF ** 2 / 3
    dq = (square[..., None] * (P @ K).square()).sum() * scale ** 2
    dk = (square * Q.square().sum(-1) * P.square().sum(-1)).sum() * scale ** 2
    return float(dq), float(dk)


def _run(m, length, d, mean):
    q, k, v, do = _make(m, d, mean)
    lens = None if length is None else [length]
    ln = None if length is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = B.sparge_cross_fwd(q, k, v, ln)
    got = B.sparge_cross_bwd(q, k, v, o, lse, do, ln, check_status=True)
    out, _ = reference(q, k, v, lens, dout=do)
    errors = [float((t.double() - out[n]).norm()) for t, n in zip(got, ("dq", "dk", "dv"))]
    return errors, [float(out[n].norm()) for n in ("dq", "dk", "dv")], _of_D(q, k, v, do, length or m)


@pytest.mark.parametrize("mean", [0, 3, 10])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m,length", [(2, None), (10, None), (64, None), (64, 2), (33, 30)])
def test_short_contexts_have_no_part_of_the_mean(m, length, d, mean):
    errors, norms, _ = _run(m, length, d, mean)
    for name, e, n in zip(("dq", "dk", "dv"), errors, norms):
        assert e <= TWO * n, (name, e / n)


@pytest.mark.parametrize("mean", [0, 1, 3, 10])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m,length", [(65, None), (128, None), (300, None), (512, None), (512, 2),
                                      (512, 30)])
def test_longer_ones_have_what_the_rounding_of_the_output_gives(m, length, d, mean):
    errors, norms, of_D = _run(m, length, d, mean)
    for name, e, n, extra in zip(("dq", "dk", "dv"), errors, norms, (*of_D, 0.0)):
        assert e <= (TWO ** 2 * n ** 2 + extra) ** 0.5, (name, e / n)
