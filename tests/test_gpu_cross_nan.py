"""NaN among the queries and the valid keys of the attention over a context: it stays where the
formula puts it, and is not taken for a row or a part without keys."""

import pytest
import torch

from block_sparse_attention_sparge_gb300 import binding as B

pytestmark = pytest.mark.gpu
NAN = float("nan")

# (B, H, N, M, d): a tile's keys at once, in parts, and query tiles that fill the machine
SHAPES = [(1, 2, 100, 33, 64), (1, 2, 300, 400, 128), (2, 1, 5, 5000, 128), (1, 3, 130, 3000, 64),
          (2, 10, 2200, 200, 128), (4, 20, 1030, 130, 64)]


def _make(shape, seed):
    b, h, n, m, d = shape
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(s, generator=g).to(torch.bfloat16).cuda()
            for s in ((b, h, n, d), (b, h, m, d), (b, h, m, d), (b, h, n, d))]


@pytest.mark.parametrize("k", range(len(SHAPES)))
def test_a_query(k):
    q, kk, v, do = _make(SHAPES[k], k)
    o, lse = B.sparge_cross_fwd(q, kk, v)
    row = min(3, q.shape[2] - 1)
    q[0, 1 % q.shape[1], row, 7] = NAN
    at = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
    at[0, 1 % q.shape[1], row] = True
    got, got_lse = B.sparge_cross_fwd(q, kk, v, check_status=True)
    assert got[at].isnan().all() and got_lse[at].isnan().all()
    assert torch.equal(got[~at], o[~at]) and torch.equal(got_lse[~at], lse[~at])
    dq, dk, dv = B.sparge_cross_bwd(q, kk, v, got, got_lse, do, check_status=True)
    assert dq[at].isnan().all() and dq[~at].isfinite().all()
    for t in (dk, dv):
        heads = at.any(-1)
        assert t[heads].isnan().all() and t[~heads].isfinite().all()


@pytest.mark.parametrize("where", [0, -1])
@pytest.mark.parametrize("k", range(len(SHAPES)))
def test_a_key_or_value(k, where):
    q, kk, v, _ = _make(SHAPES[k], k)
    o, lse = B.sparge_cross_fwd(q, kk, v)
    bad = kk.clone()
    bad[0, 0, where, 5] = NAN
    got, got_lse = B.sparge_cross_fwd(q, bad, v, check_status=True)
    assert got[0, 0].isnan().all() and got_lse[0, 0].isnan().all()
    assert torch.equal(got[1:], o[1:]) and torch.equal(got[0, 1:], o[0, 1:])
    bad = v.clone()
    bad[0, 0, where, 5] = NAN
    got, got_lse = B.sparge_cross_fwd(q, kk, bad)
    assert got[0, 0, :, 5].isnan().all() and torch.equal(got_lse, lse)
    got[0, 0, :, 5] = o[0, 0, :, 5]
    assert torch.equal(got, o)


@pytest.mark.parametrize("k", range(len(SHAPES)))
def test_infinite_scores(k):
    """exp(inf - inf): the row is NaN, as in the formula (its log-sum-exp infinite or NaN)."""
    q, kk, v, _ = _make(SHAPES[k], k)
    q[0, 0, 0], kk[0, 0, -1] = 3e30, 3e30
    got, got_lse = B.sparge_cross_fwd(q, kk, v, check_status=True)
    assert got[0, 0, 0].isnan().all() and not got_lse[0, 0, 0].isfinite()
