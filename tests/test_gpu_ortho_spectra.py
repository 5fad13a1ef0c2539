"""Orthogonalised updates of matrices with prescribed singular values: a few strong directions
and others far below them, whose errors the iteration multiplies by up to |a| a step."""

import math

import pytest
import torch

from block_sparse_attention_sparge_gb300 import binding as B
from ortho_reference import COEFF, reference

pytestmark = pytest.mark.gpu
SEEDS = 6


def _matrix(m, n, spectrum, cond, seed):
    g = torch.Generator().manual_seed(seed)
    u, v = (torch.linalg.qr(torch.randn(r, m, generator=g, dtype=torch.float64))[0] for r in (m, n))
    if spectrum == "even":
        s = torch.logspace(0, -math.log10(cond), m, dtype=torch.float64)
    else:
        s = torch.full((m,), 1 / cond, dtype=torch.float64)
        s[:{"one strong": 1, "two strong": 2}[spectrum]] = 1
    return ((u * s) @ v.T).float()


def _half(x):
    return x.half().double()


def _pair(x):
    hi = _half(x)
    return hi + _half(x - hi)


def _scheme(g, half):
    """The iteration in 64 bits with the kernels' roundings of what they multiply: X in fp16 or in
    pairs of it, scaled by a power of two near the root of the long side; A and B scaled by 256,
    their diagonals apart; X itself in pairs (fp32 in the other form, which is more)."""
    a, b, c = COEFF
    keep = _half if half else _pair
    kx = 2.0 ** round(math.log2(g.shape[1]) / 2)
    x = g.double()
    x = x / (x.norm() + 1e-7)
    for _ in range(5):
        x = _pair(x * kx) / kx if half else x.float().double()
        y = keep(x * kx) / kx
        d = x.square().sum(1)
        off = 1 - torch.eye(len(x), dtype=torch.float64)
        e = keep(256 * (y @ y.T) * off) / 256
        ee = e @ e
        f = keep(256 * (e * (b + c * (d[:, None] + d)) + c * ee) * off) / 256
        x = (a + b * d + c * (d * d + ee.diagonal()))[:, None] * x + f @ y
    return x


@pytest.mark.parametrize("spectrum", ["even", "one strong", "two strong"])
@pytest.mark.parametrize("m,n", [(2, 2), (2, 512), (4, 4), (4, 512), (16, 16), (16, 512), (64, 256),
                                 (128, 128)])
def test_no_further_off_than_the_roundings_of_the_factors(m, n, spectrum):
    """The largest error of six matrices, in the 2-norm, against that of the scheme's roundings
    alone. (Which way a value next to a border is rounded depends on sums in fp32, so the errors
    are not the same ones: twice the largest, and what the tests of spread matrices allow.)
    Beside pairs of fp16, 2^-22 of a value, there is what the tensor cores take from a sum: up
    to 2^-23 of it at each of the up to 16 additions of a chunk of four steps, 2^-19, which is
    eight times as much."""
    for cond in (1e2, 1e4, 1e6):
        for half, floor, times in ((True, 2.0 ** -8.5, 2), (False, 2.0 ** -17, 8)):
            mine, theirs = [], []
            for seed in range(SEEDS):
                g = _matrix(m, n, spectrum, cond, seed)
                want = reference(g)
                o = B.sparge_orthogonalize([g.cuda()], half=half)[0].cpu().double()
                mine.append(float((o - want).norm() / want.norm()))
                theirs.append(float((_scheme(g, half) - want).norm() / want.norm()))
            assert max(mine) <= times * max(theirs) + floor, (cond, half, mine, theirs)
            # as the header has it
            assert max(mine) <= (2.0 ** -4 if half else 2.0 ** -14)
