"""Gradient kernels called many times: no bounded wait runs out (each would cost two seconds and
the call's results), whatever the warps' order."""

import pytest
import torch

from block_sparse_attention_sparge_gb300 import binding as B

pytestmark = pytest.mark.gpu


def _rand(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(torch.bfloat16).cuda()


def _many(call, outs, status, calls=6000):
    call()
    want = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(20):
            call()
    for _ in range(calls // 20):
        graph.replay()
    torch.cuda.synchronize()
    assert int(status) == 0
    for a, b in zip(outs, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("shape", [(1, 12, 5000, 3, 64), (2, 3, 700, 300, 128), (3, 8, 900, 257, 64)])
def test_over_a_context(shape):
    b, h, n, m, d = shape
    q, k, v, do = _rand(1, b, h, n, d), _rand(2, b, h, m, d), _rand(3, b, h, m, d), _rand(4, b, h, n, d)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = B.sparge_cross_fwd(q, k, v)
    outs = [torch.empty_like(t) for t in (q, k, v)]
    _many(lambda: B.sparge_cross_bwd(q, k, v, o, lse, do, out=outs, status=status), outs, status)


@pytest.mark.parametrize("n,d", [(1000, 64), (2500, 128)])
def test_block_sparse(n, d):
    q, k, v, do = (_rand(i, 1, 3, n, d) for i in range(4))
    mask = B.sparge_mask(q, k, 0.3, 0.5)
    lists = mask["row_idx"], mask["row_cnt"], mask["col_idx"], mask["col_cnt"]
    o, lse = B.sparge_attn_fwd(q, k, v, *lists[:2])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = [torch.empty_like(t) for t in (q, k, v)]

    def call():
        for t, g in zip(outs, B.sparge_attn_bwd(q, k, v, o, lse, do, *lists, status=status)):
            t.copy_(g)

    _many(call, outs, status)
