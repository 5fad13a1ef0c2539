"""Outputs that the caller gives to sparge_heads_fwd and sparge_heads_bwd: what
autograd is told of them, and where they may lie."""

import pytest
import torch

from block_sparse_attention_sparge_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def _rand(seed, *shape, dtype=BF):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DEV, dtype)


def test_autograd_notices_that_an_output_was_written():
    b, n, h, d = 1, 9, 2, 64
    q, k = _rand(1, b, n, h, d), _rand(2, b, n, h, d)
    leaf = torch.ones((), device=DEV, requires_grad=True)
    out, free = _rand(3, b, h, n, d), _rand(4, b, h, n, d)
    kept = (leaf * out).sum()  # keeps out for its backward
    before = free._version
    B.sparge_heads_fwd(q, None, None, out=(out, free, None))
    assert free._version == before  # not written: there is no k
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        kept.backward()

    buf = _rand(5, b, n, 2 * h * d)
    kept = (leaf * buf).sum()
    parts = [t.unflatten(-1, (h, d)) for t in buf.chunk(2, -1)]
    B.sparge_heads_bwd(None, _rand(6, b, h, n, d), None, None, k, out=(None, parts[1], None))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        kept.backward()
    (leaf * buf).sum().backward()  # of what it holds now
    assert leaf.grad.isfinite()


def _refused(call):
    with pytest.raises(B.SpargeError) as e:
        call()
    assert e.value.code == B.SPARGE_ERR_INVALID_ARG


def test_outputs_that_share_memory_are_refused():
    """Outputs over one another in part, over themselves, over an input."""
    b, n, h, d = 2, 9, 2, 64
    size = b * n * h * d
    q, k = _rand(1, b, n, h, d), _rand(2, b, n, h, d)
    buf = _rand(3, 4 * size)
    a, c = buf[:size].view(b, h, n, d), buf[size - 8:][:size].view(b, h, n, d)
    before = buf.clone()
    _refused(lambda: B.sparge_heads_fwd(q, k, None, out=(a, c, None)))
    _refused(lambda: B.sparge_heads_fwd(a.view(b, n, h, d), k, None, out=(None, c, None)))
    _refused(lambda: B.sparge_heads_fwd(a.view(b, n, h, d), out=(a, None, None)))
    dq, dk = _rand(4, b, h, n, d), _rand(5, b, h, n, d)
    # slices of one buffer, the second half a head too early
    rows = buf[:b * n * 3 * h * d].view(b, n, 3 * h * d)
    parts = [rows[..., at:at + h * d].unflatten(-1, (h, d)) for at in (0, h * d - 32)]
    _refused(lambda: B.sparge_heads_bwd(dq, dk, out=(*parts, None)))
    # samples that begin inside one another
    own = buf.as_strided((b, n, h, d), (4 * h * d, h * d, d, 1))
    _refused(lambda: B.sparge_heads_bwd(dq, out=(own, None, None)))
    # over the gradient that is read, over another part's input
    _refused(lambda: B.sparge_heads_bwd(a, out=(a.view(b, n, h, d), None, None)))
    _refused(lambda: B.sparge_heads_bwd(dq, dk, None, q, k, norm="head", out=(k, q, None)))
    torch.cuda.synchronize()
    assert torch.equal(buf, before)


@pytest.mark.parametrize("norm", ["token", "head"])
@pytest.mark.parametrize("h,dtype", [(3, BF), (3, F32), (24, BF), (24, F32)])
def test_gradients_in_place_of_their_inputs(norm, h, dtype):
    b, n, d = 2, 77, 128
    q, k = _rand(1, b, n, h, d, dtype=dtype), _rand(2, b, n, h, d, dtype=dtype)
    grads = [_rand(3 + i, b, h, n, d) for i in range(3)]
    w = _rand(7, h * d if norm == "token" else d, dtype=F32)
    how = dict(norm=norm, q_weight=w, k_weight=w)
    want = B.sparge_heads_bwd(*grads, q, k, **how)
    got = B.sparge_heads_bwd(*grads, q, k, out=(q, k, None), **how)
    assert got[0] is q and got[1] is k
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_one_head_in_place_and_orders_that_lie_apart():
    b, n, d = 2, 33, 64
    x = _rand(1, b, n, 1, d)
    want = B.sparge_heads_fwd(x, norm="head")[0]
    assert torch.equal(B.sparge_heads_fwd(x, norm="head", out=(x.view(b, 1, n, d), None, None))[0],
                       want)
    # parts of different head counts as slices; tokens outermost; every second token
    g = [_rand(2 + i, b, h, n, d) for i, h in enumerate((4, 1, 2))]
    want = B.sparge_heads_bwd(*g)[:3]
    buf = torch.zeros(b, n, 7 * d, dtype=BF, device=DEV)
    sliced = [t.unflatten(-1, (-1, d)) for t in buf.split((4 * d, d, 2 * d), -1)]
    outer = [torch.zeros(n, t.shape[1], b, d, dtype=BF, device=DEV).permute(2, 0, 1, 3) for t in g]
    both = torch.zeros(b, 2 * n, 4, d, dtype=BF, device=DEV)
    for out in (sliced, outer, (both[:, ::2], both[:, 1::2, :1], both[:, 1::2, 1:3])):
        for got, ref in zip(B.sparge_heads_bwd(*g, out=out), want):
            assert torch.equal(got, ref)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("n,h", [(77, 1), (1, 5), (1, 40)])
def test_gradients_in_place_of_the_gradients_they_come_from(n, h, interleaved):
    """One head, or one token a sample: both layouts are the same."""
    b, d = 203, 128
    g = [_rand(i, b, h, n, d) for i in range(3)]
    q, k = _rand(5, b, n, h, d), _rand(6, b, n, h, d)
    pos = torch.randint(0, 99, (b, n, 3), generator=torch.Generator().manual_seed(7))
    how = dict(norm="head", pos=pos.to(DEV, torch.int32),
               rope=B.RopeAxes(d, (22, 21, 21), interleaved=interleaved))
    want = B.sparge_heads_bwd(*g, q, k, **how)[:3]
    got = B.sparge_heads_bwd(*g, q, k, out=[t.view(b, n, h, d) for t in g], **how)
    for x, y in zip(got, want):
        assert torch.equal(x, y)
