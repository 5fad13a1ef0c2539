"""Lists of matrices of both forms: refused as a whole before anything is written."""

import pytest
import torch

from block_sparse_attention_sparge_gb300 import binding as B
from ortho_reference import check, reference

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _rand(seed, *shape, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


def test_a_result_on_a_gradient_of_the_other_form():
    a, b = _rand(1, 40, 64), _rand(2, 40, 64, dtype=BF)
    on_a = a.view(BF)[:, :64]
    keep = a.clone()
    for mats, out in (([b, a], [on_a, torch.empty_like(a)]), ([a, b], [torch.empty_like(a), on_a])):
        with pytest.raises(B.SpargeError) as e:
            B.sparge_orthogonalize(mats, out=out)
        assert e.value.code == B.SPARGE_ERR_INVALID_ARG and torch.equal(a, keep)


def test_a_momentum_of_two_weights():
    ws = [_rand(1, 40, 64), _rand(2, 40, 64, dtype=BF)]
    gs, m = [_rand(3, 40, 64), _rand(4, 40, 64)], _rand(5, 40, 64)
    keep = [t.clone() for t in (*ws, m)]
    with pytest.raises(B.SpargeError):
        B.sparge_muon_step(ws, gs, [m, m], 0.1)
    assert all(torch.equal(a, b) for a, b in zip((*ws, m), keep))


def test_one_that_is_refused_leaves_the_others():
    """Whatever the order and the form of the bad one: a workspace that is too small for either."""
    small, large = _rand(1, 20, 30, dtype=BF), _rand(2, 200, 300)
    for mats in ([small, large], [large, small], [small.float(), large.to(BF)]):
        own = [m.clone() for m in mats]
        with pytest.raises(B.SpargeError) as e:
            # (enough for a 20 x 30 one of either form, 0.5 MB, not for the other)
            B.sparge_orthogonalize(own, out=own, workspace=torch.empty(600_000, dtype=torch.uint8,
                                                                      device="cuda"))
        assert e.value.code == B.SPARGE_ERR_WORKSPACE
        assert all(torch.equal(a, b) for a, b in zip(own, mats))


def test_one_workspace_for_both_forms():
    mats = [_rand(i, 60 + 40 * i, 150, dtype=t) for i, t in enumerate((BF, F32, BF, F32))]
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    for kw in ({}, dict(workspace=ws)):
        for g, o in zip(mats, B.sparge_orthogonalize(mats, check_status=True, **kw)):
            check(o, reference(g), g.dtype == BF)
