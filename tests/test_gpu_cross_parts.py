"""Attention over a context where its sums are cut into parts: gradients of samples of other
lengths (which may change under a captured call), few queries over keys of any number; and
narrow heads over query tiles that fill the machine."""

import pytest
import torch

from block_sparse_attention_sparge_gb300 import binding as B
from cross_reference import check, reference

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _make(shape, seed):
    b, bk, h, hk, n, m, d = shape
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(s, generator=g).to(BF).cuda()
            for s in ((b, h, n, d), (bk, hk, m, d), (bk, hk, m, d), (b, h, n, d))]


SHAPES = [
    (4, 4, 4, 2, 700, 520, 64), (4, 1, 4, 2, 700, 520, 64), (4, 4, 3, 3, 300, 600, 128),
    (4, 1, 3, 3, 300, 600, 128),
]
LENS = [[520, 519, 129, 128], [0, 0, 0, 0], [0, 0, 0, 1], [520, 0, 0, 0], [1, 2, 3, 4],
        [-7, 10000, 0, 257]]


@pytest.mark.parametrize("k", range(len(SHAPES)))
def test_lengths_that_change_under_a_captured_call(k):
    q, kk, v, do = _make(SHAPES[k], k)
    lens = torch.tensor(LENS[0], dtype=torch.int32, device="cuda")
    outs = [torch.empty_like(t) for t in (q, kk, v)]

    def both():
        o, lse = B.sparge_cross_fwd(q, kk, v, lens)
        B.sparge_cross_bwd(q, kk, v, o, lse, do, lens, out=outs)

    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for now in LENS + LENS[:1]:
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        for t in outs:
            t.fill_(9.0)
        graph.replay()
        out, lim = reference(q, kk, v, now, dout=do)
        check(outs, out, lim, ("dq", "dk", "dv"))
        o, lse = B.sparge_cross_fwd(q, kk, v, lens)
        for a, t in zip(B.sparge_cross_bwd(q, kk, v, o, lse, do, lens, check_status=True), outs):
            assert torch.equal(a, t)


def test_more_samples_than_lanes():
    shape = (70, 70, 2, 1, 130, 260, 64)
    q, kk, v, do = _make(shape, 9)
    lens = [(i * 37) % 262 - 1 for i in range(70)]
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = B.sparge_cross_fwd(q, kk, v, ln)
    out, lim = reference(q, kk, v, lens, dout=do)
    check(B.sparge_cross_bwd(q, kk, v, o, lse, do, ln), out, lim, ("dq", "dk", "dv"))


def test_full_lengths_are_no_lengths():
    q, kk, v, do = _make((2, 2, 4, 4, 1000, 300, 128), 3)
    ln = torch.full((2,), 300, dtype=torch.int32, device="cuda")
    o, lse = B.sparge_cross_fwd(q, kk, v)
    for a, b in zip(B.sparge_cross_bwd(q, kk, v, o, lse, do),
                    B.sparge_cross_bwd(q, kk, v, o, lse, do, ln)):
        assert torch.equal(a, b)


FILLED = [
    ((80, 80, 4, 4, 129, 66, 64), None),
    ((1, 1, 5, 5, 16100, 700, 64), None),
    ((14, 1, 6, 2, 1000, 400, 64), [400, 1, 0, 128, 257, 399, 3] * 2),
    ((160, 160, 4, 2, 1, 200, 64), None),
    ((130, 130, 5, 1, 2, 129, 64), [129 - (i * 7) % 130 for i in range(130)]),
]


@pytest.mark.parametrize("tokens", [True, False])
@pytest.mark.parametrize("k", range(len(FILLED)))
def test_narrow_heads_that_fill_the_machine(k, tokens):
    shape, lens = FILLED[k]
    q, kk, v, _ = _make(shape, k)
    if tokens:
        q, kk, v = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, kk, v))
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda") if lens else None
    o, lse = B.sparge_cross_fwd(q, kk, v, ln, check_status=True)
    out, lim = reference(q, kk, v, lens)
    check((o, lse), out, lim, ("o", "lse"))
    if lens:  # what stands behind the lengths is not used
        for t in (kk, v):
            for b in range(t.shape[0]):
                t[b, :, max(lens) if t.shape[0] == 1 else lens[b]:] = float("nan")
        again = B.sparge_cross_fwd(q, kk, v, ln)
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m", [640, 1000, 1153, 1600, 2111, 6000])
def test_few_queries_in_parts_or_not(m, d):
    for h, n in ((1, 5), (4, 300), (8, 2048)):
        q, kk, v, _ = _make((2, 2, h, h, n, m, d), m)
        lens = [m, m // 3]
        ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
        got = B.sparge_cross_fwd(q, kk, v, ln, check_status=True)
        out, lim = reference(q, kk, v, lens)
        check(got, out, lim, ("o", "lse"))
