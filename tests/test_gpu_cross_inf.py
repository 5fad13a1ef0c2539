"""Scores of minus infinity in the attention over a context: keys masked through a channel (of
-inf, or of products that leave fp32) have P = 0 wherever they stand, and a row that has no other
keys is a row without keys."""

import math

import pytest
import torch

from block_sparse_attention_sparge_gb300 import binding as B
from cross_reference import FP32, HALF, check

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

# (B, H, N, M, d): a tile's keys at once, in parts, and query tiles that fill the machine
SHAPES = [(1, 2, 100, 200, 64), (1, 2, 300, 400, 128), (2, 1, 5, 5000, 128), (1, 3, 130, 3000, 64),
          (2, 10, 2200, 200, 128), (4, 20, 1030, 130, 64)]


def _masked(name, m):
    at = torch.arange(m)
    return {"first": at < 16, "step": at < 64, "steps": at < 128, "all but the last": at < m - 1,
            "every other step": at // 64 % 2 == 0, "last": at >= m - 20, "scattered": at * 7 % 5 < 3,
            "first part": at < m // 2, "all": at >= 0}[name]


def _make(shape, name, how, level, rows, seed, scale=None):
    """q, k, v, do and the mask [N, M]. Channel 0 masks the keys of ``name`` for the queries of
    ``rows``; channel 1 shifts all scores to about ``level``. ``how``: the masked keys' channel 0."""
    b, h, n, m, d = shape
    g = torch.Generator().manual_seed(seed)
    q, k, v, do = (torch.randn(s, generator=g) for s in
                   ((b, h, n, d), (b, h, m, d), (b, h, m, d), (b, h, n, d)))
    scale = scale or d ** -0.5
    keys, queries = _masked(name, m), torch.ones(n, dtype=torch.bool)
    if rows == "half":
        queries = torch.arange(n) % 2 == 0
    finite = math.isfinite(how)
    # (an infinity times 0 would be NaN, so all queries have it there)
    q[..., 0] = (queries.float() * 1e30) if finite else 1.0
    k[..., 0] = torch.where(keys, torch.tensor(how), torch.tensor(0.0))
    q[..., 1], k[..., 1] = 1.0, level / scale
    return [t.to(BF).cuda() for t in (q, k, v, do)], (queries[:, None] & keys).cuda()


def _reference(q, k, v, do, mask, scale=None):
    d = q.shape[-1]
    scale = scale or d ** -0.5
    Q, K, V, G = (t.double() for t in (q, k, v, do))
    Q0, K0 = Q.clone(), K.clone()
    Q0[..., 0] = 0
    K0[..., 0] = 0
    s = (scale * Q0 @ K0.transpose(-1, -2)).masked_fill(mask, -math.inf)
    lse = s.logsumexp(-1)
    P = (s - lse.masked_fill(lse == -math.inf, 0.0)[..., None]).exp()
    o = P @ V
    size = P @ V.abs()
    lim_o = HALF * (size + o.abs()) + FP32 * size
    dS = P * (G @ V.transpose(-1, -2) - (G * o).sum(-1, keepdim=True))
    off = (HALF * dS.abs() + P * (G.abs() * lim_o).sum(-1, keepdim=True)
           + FP32 * P * (G.abs() @ V.abs().transpose(-1, -2) + (G * o).abs().sum(-1, keepdim=True)))
    dk, off_k = ((x.transpose(-1, -2) @ y) * scale for x, y in ((dS, Q), (off, Q.abs())))
    dq, off_q = ((x @ y) * scale for x, y in ((dS, K), (off, K.abs())))
    dv = P.transpose(-1, -2) @ G
    out = {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    lim = {"o": lim_o, "dq": off_q + HALF * dq.abs(), "dk": off_k + HALF * dk.abs(),
           "dv": (HALF + FP32) * (P.transpose(-1, -2) @ G.abs()) + HALF * dv.abs()}
    return out, lim


NAMES = ["first", "step", "steps", "all but the last", "every other step", "last", "scattered",
         "first part", "all"]


@pytest.mark.parametrize("how", [-math.inf, -1e30])
@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("k", range(len(SHAPES)))
def test_masked_keys(k, name, how):
    for level in (0.0, -375.0, 375.0):
        (q, kk, v, do), mask = _make(SHAPES[k], name, how, level, "all", k)
        o, lse = B.sparge_cross_fwd(q, kk, v, check_status=True)
        out, lim = _reference(q, kk, v, do, mask)
        check((o, lse), out, lim, ("o", "lse"))


@pytest.mark.parametrize("k", range(len(SHAPES)))
def test_masked_keys_under_a_negative_scale(k):
    (q, kk, v, do), mask = _make(SHAPES[k], "step", math.inf, 20.0, "all", k, -0.1)
    got = B.sparge_cross_fwd(q, kk, v, softmax_scale=-0.1, check_status=True)
    out, lim = _reference(q, kk, v, do, mask, -0.1)
    check(got, out, lim, ("o", "lse"))


@pytest.mark.parametrize("rows", ["all", "half"])
@pytest.mark.parametrize("name", ["step", "every other step", "all but the last", "all"])
@pytest.mark.parametrize("shape", SHAPES + [(1, 2, 150, 40, 64), (1, 1, 150, 64, 128)])
def test_gradients_of_masked_keys(shape, name, rows):
    """Rows whose keys are all masked add nothing to any gradient."""
    (q, kk, v, do), mask = _make(shape, name, -1e30, 0.0, rows, 3)
    o, lse = B.sparge_cross_fwd(q, kk, v)
    got = B.sparge_cross_bwd(q, kk, v, o, lse, do, check_status=True)
    out, lim = _reference(q, kk, v, do, mask)
    # Channel 0 of dQ is -1e30 scale times the sum of dS over the masked keys. In a row that
    # they are not masked for, that is minus the sum over the others (all of them add up to 0):
    # with one other of 130 keys, 129 terms of the size of the one that is left, each rounded
    # (2^-9 / sqrt(3), sqrt(129) of them), and D's rounding 129 times over: 0.01 and more of
    # the result. So it has its bound alone, element by element, and no 2-norm beside it.
    e = (got[0][..., 0].double() - out["dq"][..., 0]).abs()
    assert (e <= lim["dq"][..., 0]).all()
    check((got[0][..., 1:],), *({"dq": t["dq"][..., 1:]} for t in (out, lim)), ("dq",))
    check(got[1:], out, lim, ("dk", "dv"))
    alone = mask.all(-1)
    assert (got[0][:, :, alone] == 0).all()
