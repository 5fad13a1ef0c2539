"""Weight, gate, scale and shift gradients as sums over rows in which no row may
be lost or counted twice.

Residual norm: small whole numbers, whose sums fp32 holds exactly in any order
(all of them stay below 2^24), so the gradients match bit for bit.  Head layout:
the terms are +-1 up to the rounding of 1 / rms (two products and a reciprocal root
of at most two steps: 8 * 2^-24), and a sum's bound counts its longest chain of
additions instead of one for every row: at these sizes at most 24 tokens of a
slot, 2 vectors and 3 steps over lanes, 20 warps or 6 slots of a CTA, 16 partial
rows of a slice and 32 slices, in all below 128."""

import pytest
import torch

import block_reference as R
from block_sparse_attention_sparge_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
TYPES = [(BF, BF), (F32, BF), (F32, F32)]
CHAIN = (8 + 128) * R.U


def _ints(g, *shape, dtype, most=3):
    return torch.randint(-most, most + 1, shape, generator=g).to(DEV, dtype)


def _rows(t, groups):
    """Sums of [rows, C] over each group's rows, in whole numbers."""
    t = t.long() if t.dtype != torch.int64 else t
    return t.unflatten(0, (groups, -1)).sum(1).double().cpu()


# rows, groups: odd counts, remainders of one row, one row a group, few groups
ROWS = [(1, 1), (9001, 1), (9000, 3), (2002, 2002), (4097 * 3, 3)]


@pytest.mark.parametrize("tx,tb", TYPES)
@pytest.mark.parametrize("post", [False, True], ids=["plain", "post"])
@pytest.mark.parametrize("c", [8, 64, 264, 1536, 2560, 5120, 5376])
def test_residual_norm_sums_are_exact(c, post, tx, tb):
    g = torch.Generator().manual_seed(c)
    for rows, groups in ROWS:
        rows = min(rows, 3_000_000 // c // groups * groups) if rows > 2 * groups else rows
        if rows * c > 20_000_000:
            continue
        x, dy = (_ints(g, 1, rows, c, dtype=tx) for _ in range(2))
        b, dh = (_ints(g, 1, rows, c, dtype=tb) for _ in range(2))
        gate, scale, shift = (_ints(g, 1, groups, c, dtype=F32, most=2) for _ in range(3))
        w = _ints(g, c, dtype=F32, most=2) if post else None
        # statistics as a forward might have left them: nothing is scaled
        stats = torch.ones(3, rows, device=DEV)
        per = rows // groups
        n = b.float() * (w if post else 1.0)
        y = x.float() + gate.repeat_interleave(per, 1) * n
        how = dict(stats=stats, norm="rms", post_weight=w)
        got = B.sparge_resnorm_bwd(dy, dh, x, b, gate, scale, shift, **how)
        assert torch.equal(R.f64(got[3])[0], _rows((dh.float() * y)[0], groups)), (rows, groups)
        assert torch.equal(R.f64(got[4])[0], _rows(dh[0], groups)), (rows, groups)
        # without a gradient behind the norm, dx is dy
        for more in (torch.zeros_like(dh), None):
            got = B.sparge_resnorm_bwd(dy, more, x, b, gate, scale, shift, **how)
            assert torch.equal(got[0], dy)
            assert torch.equal(R.f64(got[2])[0], _rows((dy.float() * n)[0], groups)), (rows, groups)
            assert not got[3].any() and not got[4].any()
            if post:
                e = dy.float() * gate.repeat_interleave(per, 1) * b.float()
                assert torch.equal(R.f64(got[5]), _rows(e[0], 1)[0]), (rows, groups)


def test_one_row_of_each_beside_rows_for_groups():
    """A gate for each frame, scale and shift of the model: sums by item and by
    slot in one call."""
    g = torch.Generator().manual_seed(1)
    rows, c, f = 7 * 301, 1536, 7
    x, dy, b, dh = (_ints(g, 1, rows, c, dtype=BF) for _ in range(4))
    gate = _ints(g, 1, f, c, dtype=F32, most=2)
    scale, shift = (_ints(g, c, dtype=F32, most=2) for _ in range(2))
    stats = torch.ones(3, rows, device=DEV)
    got = B.sparge_resnorm_bwd(dy, dh, x, b, gate, scale, shift, stats, norm="rms")
    y = x.float() + gate.repeat_interleave(rows // f, 1) * b.float()
    assert torch.equal(R.f64(got[3]), _rows((dh.float() * y)[0], 1)[0])
    assert torch.equal(R.f64(got[4]), _rows(dh[0], 1)[0])
    got = B.sparge_resnorm_bwd(dy, torch.zeros_like(dh), x, b, gate, scale, shift, stats,
                               norm="rms")
    assert torch.equal(R.f64(got[2])[0], _rows((dy.float() * b.float())[0], f))


@pytest.mark.parametrize("norm", ["token", "head"])
@pytest.mark.parametrize("b,n,h,d,dtype", [
    (6000, 1, 2, 64, BF), (1, 6001, 1, 64, F32), (2, 3001, 12, 128, BF), (3, 1001, 12, 128, F32),
    (1, 2003, 20, 128, BF), (1, 1501, 40, 128, F32), (1, 1501, 40, 128, BF), (1, 701, 64, 128, BF),
    (2, 351, 42, 128, F32), (1, 1, 7, 64, BF),
])
def test_head_layout_weight_sums_miss_no_row(b, n, h, d, dtype, norm):
    g = torch.Generator().manual_seed(n)
    sign = lambda: (torch.randint(0, 2, (b, n, h, d), generator=g) * 2 - 1)  # noqa: E731
    q, k, sq, sk = sign(), sign(), sign(), sign()
    dq, dk = (s.transpose(1, 2).contiguous().to(DEV, BF) for s in (sq, sk))
    width = h * d if norm == "token" else d
    w = torch.ones(width, device=DEV)
    for heads in ((dq, dk, dq), (dq, dk, None)):  # V beside them, or not
        got = B.sparge_heads_bwd(*heads, q.to(DEV, dtype), k.to(DEV, dtype), norm=norm, q_weight=w,
                                 k_weight=w, eps=0.0)
        for x, s, dw in ((q, sq, got[3]), (k, sk, got[4])):
            over = (0, 1) if norm == "token" else (0, 1, 2)
            want = (x * s).sum(over).flatten().double()
            terms = b * n * (1 if norm == "token" else h)
            assert CHAIN * terms < 1.0  # less than one term
            R.check(dw, want, torch.full_like(want, CHAIN * terms))
