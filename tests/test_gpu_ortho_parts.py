"""Orthogonalised updates whose long sides are summed in parts, against 64 bits."""

import pytest
import torch

from block_sparse_attention_sparge_gb300 import binding as B
from ortho_reference import check, reference

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _rand(seed, *shape, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


SHAPES = [
    [(1, 65536)], [(16, 5120)], [(4100, 100)], [(128, 20001)], [(129, 9000)], [(8000, 300)],
    [(640, 2100)], [(3, 385)], [(3, 257)],
    [(1536, 24), (16, 5120), (700, 333), (64, 1001), (1, 77), (129, 129)],
    [(130, 7000), (20, 20), (6000, 20)], [(5, 3000)] * 40,
]


@pytest.mark.parametrize("k", range(len(SHAPES)))
@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_sides(k, dtype):
    gs = [_rand(50 * k + i, *s, dtype=dtype) for i, s in enumerate(SHAPES[k])]
    outs = B.sparge_orthogonalize(gs, check_status=True)
    for g, o in zip(gs, outs):
        check(o, reference(g), dtype == BF)
    # the parts are added in their order, whichever comes last
    for _ in range(3):
        for a, o in zip(B.sparge_orthogonalize(gs), outs):
            assert torch.equal(a, o)


@pytest.mark.parametrize("half", [True, False])
def test_one_workspace_for_lists_of_other_plans(half):
    """Counters lie elsewhere for each list, and what an earlier one left there does not matter."""
    lists = [[_rand(10 * k + i, *s) for i, s in enumerate(shapes)]
             for k, shapes in enumerate(([(16, 5120)], [(300, 300)], [(130, 7000), (20, 2000)]))]
    ws = torch.full((256 << 20,), 0xA5, dtype=torch.uint8, device="cuda")
    for gs in lists * 2:
        for g, o in zip(gs, B.sparge_orthogonalize(gs, half=half, workspace=ws, check_status=True)):
            check(o, reference(g), half)


def test_captured_and_replayed():
    gs = [_rand(1, 40, 6000), _rand(2, 200, 1500)]
    outs = [torch.empty_like(g) for g in gs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.sparge_orthogonalize(gs, out=outs)
    for seed in (3, 4, 5):
        for i, g in enumerate(gs):
            g.copy_(_rand(10 * seed + i, *g.shape))
        graph.replay()
        for g, o in zip(gs, outs):
            check(o, reference(g), False)


@pytest.mark.parametrize("half", [True, False])
def test_nan_stays_in_its_matrix(half):
    bad, good = _rand(1, 60, 4000), _rand(2, 60, 4000)
    bad[59, 3999] = float("nan")
    outs = B.sparge_orthogonalize([bad, good], half=half)
    assert outs[0].isnan().all()
    check(outs[1], reference(good), half)
