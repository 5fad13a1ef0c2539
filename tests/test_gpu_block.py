"""The operators around the attention used together: autograd, a stack of
residual blocks with rotary positions, norms and modulation, and a fine-tuning
step with clipping, against plain 64-bit torch."""

import pytest
import torch

import block_reference as R
from block_sparse_attention_sparge_gb300 import binding as B
from block_sparse_attention_sparge_gb300 import train
from helpers import GRAD_REL_L2, O_REL_L2, rel_l2, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def _rand(g, *shape, dtype=F32, std=1.0, mean=0.0, grad=False):
    return (torch.randn(shape, generator=g) * std + mean).to(DEV, dtype).requires_grad_(grad)


def _pairs(d):
    return (d // 2 - 2 * (d // 6), d // 6, d // 6)


@pytest.mark.parametrize("norm", ["token", "head", None])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_qkv_heads_autograd(norm, dtype):
    b, n, h, d = 2, 31, 3, 64
    g = torch.Generator().manual_seed(1)
    qkv = _rand(g, b, n, 3 * h * d, dtype=dtype, grad=True)
    width = {"token": h * d, "head": d, None: 0}[norm]
    wq, wk = ((_rand(g, width, std=0.2, mean=1.0, grad=True) if width else None) for _ in range(2))
    grid = torch.tensor([[2, 3, 5], [1, 4, 4]], dtype=torch.int32)
    rope = B.RopeAxes(d, _pairs(d))
    parts = [t.unflatten(-1, (h, d)) for t in qkv.chunk(3, -1)]
    out = train.qkv_heads(*parts, rope, grid.to(DEV), None, norm, wq, wk)
    douts = [_rand(g, b, h, n, d, dtype=BF) for _ in range(3)]
    torch.autograd.backward(out, douts)
    cs = R.angles(R.positions(b, n, grid), _pairs(d), d)
    for i, w in ((0, wq), (1, wk)):
        x = R.f64(parts[i])
        y, bound = R.heads_fwd(x, R.f64(w), norm, cs, True)
        R.check(out[i], y, bound)
        dx, bound, dw, dwb = R.heads_bwd(R.f64(douts[i]), x, R.f64(w), norm, cs, True)
        R.check(qkv.grad.chunk(3, -1)[i].unflatten(-1, (h, d)), dx, bound)
        if norm:
            R.check(w.grad, dw, dwb)
    assert torch.equal(qkv.grad.chunk(3, -1)[2].unflatten(-1, (h, d)),
                       douts[2].transpose(1, 2).to(dtype))


def test_qkv_heads_with_unused_outputs_and_constant_inputs():
    g = torch.Generator().manual_seed(2)
    q, k, v = (_rand(g, 1, 9, 2, 64, grad=i != 1) for i in range(3))
    w = _rand(g, 64, mean=1.0, grad=True)
    oq, ok, ov = train.qkv_heads(q, k, v, norm="head", q_weight=w, k_weight=w.detach())
    ok.detach()
    (ov.float() * 2).sum().backward()
    assert q.grad is None and w.grad is None and torch.equal(v.grad, torch.full_like(v, 2.0))
    q.grad = v.grad = None
    oq, ok, ov = train.qkv_heads(q, k, v, norm="head", q_weight=w, k_weight=w)
    (oq.float().sum() + ok.float().sum()).backward()
    assert q.grad is not None and k.grad is None and v.grad is None
    one = torch.ones(1, 2, 9, 64, dtype=torch.float64)
    _, _, dq, bq = R.heads_bwd(one, R.f64(q), R.f64(w), "head", None, True)
    _, _, dk, bk = R.heads_bwd(one, R.f64(k), R.f64(w), "head", None, True)
    R.check(w.grad, dq + dk, bq + bk + 2.0 ** -23 * (dq.abs() + dk.abs()))
    k2 = k.detach().requires_grad_(True)
    got = torch.autograd.grad(train.qkv_heads(k=k2)[1].float().sum(), k2)[0]
    assert torch.equal(got, torch.ones_like(k2))


@pytest.mark.parametrize("tx,tb", [(BF, BF), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("norm", ["layer", "rms"])
def test_residual_norm_autograd(norm, tx, tb):
    b, n, c, f = 2, 12, 192, 3
    g = torch.Generator().manual_seed(3)
    x, br = _rand(g, b, n, c, dtype=tx, grad=True), _rand(g, b, n, c, dtype=tb, grad=True)
    table = _rand(g, b, f, 3, c, std=0.3, grad=True)
    post = _rand(g, c, std=0.2, mean=1.0, grad=True)
    y, h = train.residual_norm(x, br, table[:, :, 2], table[:, :, 1], table[:, :, 0], norm,
                               post_weight=post)
    dy, dh = _rand(g, b, n, c, dtype=tx), _rand(g, b, n, c, dtype=tb)
    torch.autograd.backward([y, h], [dy, dh])
    t = R.f64(table)
    ref = R.Resnorm(R.f64(x), R.f64(br), t[:, :, 2], t[:, :, 1], t[:, :, 0], norm, True,
                    R.f64(post))
    R.check(y, ref.y, ref.y_bound())
    R.check(h, ref.h, ref.h_bound())
    want = ref.backward(R.f64(dy), R.f64(dh))
    for name, got in (("dx", x.grad), ("dbranch", br.grad), ("dshift", table.grad[:, :, 0]),
                      ("dscale", table.grad[:, :, 1]), ("dgate", table.grad[:, :, 2]),
                      ("dpost", post.grad)):
        R.check(got, *want[name], name)


def test_residual_norm_autograd_of_its_parts():
    g = torch.Generator().manual_seed(4)
    x, br = _rand(g, 7, 64, grad=True), _rand(g, 7, 64, grad=True)
    w, bias = _rand(g, 64, mean=1.0, grad=True), _rand(g, 64, grad=True)
    y, h = train.residual_norm(x, scale=w, shift=bias, unit_offset=False)
    assert y is x
    h.sum().backward()
    ref = R.Resnorm(R.f64(x)[None], None, None, R.f64(w), R.f64(bias), unit=False)
    want = ref.backward(None, torch.ones(1, 7, 64, dtype=torch.float64))
    R.check(x.grad[None], *want["dx"])
    R.check(w.grad, *want["dscale"])
    R.check(bias.grad, *want["dshift"])
    x.grad = None
    y, h = train.residual_norm(x, br, norm=None)
    assert h is None
    y.sum().backward()
    assert torch.equal(x.grad, torch.ones_like(x)) and torch.equal(br.grad, torch.ones_like(br))
    y, h = train.residual_norm(x, br)
    y.detach()
    with pytest.raises(RuntimeError):  # the backward has no gradient of its own
        gx = torch.autograd.grad(h.sum(), x, create_graph=True)[0]
        gx.sum().backward()


class Plain64:
    """The stack in 64 bits, with dense attention."""

    def __init__(self, stack, grid, d):
        self.blocks = [{k: R.f64(v).requires_grad_(True) for k, v in b.named_parameters()}
                       for b in stack.blocks]
        self.kind = [(b.norm, b.qk_norm, b.rope.interleaved) for b in stack.blocks]
        self.grid, self.d = grid, d

    def __call__(self, x, modulation):
        b, n, c = x.shape
        f = modulation.shape[1]
        cs = R.angles(R.positions(b, n, self.grid), _pairs(self.d), self.d)
        for i, (p, (norm, qk, inter)) in enumerate(zip(self.blocks, self.kind)):
            shift, scale, gate = (modulation[:, :, i, k].repeat_interleave(n // f, 1)
                                  for k in range(3))
            z = x - x.mean(-1, keepdim=True) if norm == "layer" else x
            z = z * (z.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
            h = z * (1 + scale) + shift
            heads = []
            for w, nw in (("wq", "norm_q"), ("wk", "norm_k"), ("wv", None)):
                t = (h @ p[w]).unflatten(-1, (-1, self.d))
                if nw:
                    t = R.heads_fwd(t, p[nw], qk, cs, inter)[0]
                else:
                    t = t.transpose(1, 2)
                heads.append(t)
            q, k, v = heads
            a = torch.softmax(q @ k.transpose(-1, -2) * self.d ** -0.5, -1) @ v
            x = x + gate * (a.transpose(1, 2).flatten(2) @ p["wo"])
        return x


def _stack(c, h, d, seed=5):
    gen = torch.Generator().manual_seed(seed)
    kinds = (("layer", "token", True), ("rms", "head", False))
    return train.BlockStack([train.AttentionBlock(c, h, d, generator=gen,
                                                  rope=B.RopeAxes(d, _pairs(d), interleaved=i),
                                                  qk_norm=q, norm=n) for n, q, i in kinds])


def test_stack_of_blocks_runs_and_has_the_gradients_of_its_formula():
    c, h, d, b, n, f = 128, 2, 64, 2, 150, 3
    stack = _stack(c, h, d)
    grid = torch.tensor([[3, 5, 10], [2, 5, 10]], dtype=torch.int32)
    g = torch.Generator().manual_seed(6)
    x = _rand(g, b, n, c, grad=True)
    modulation = _rand(g, b, f, 2, 3, c, std=0.3, grad=True)
    y = stack(x, grid.to(DEV), modulation)
    w = _rand(g, b, n, c)
    (y * w).sum().backward()
    plain = Plain64(stack, grid, d)
    x64, m64 = R.f64(x).requires_grad_(True), R.f64(modulation).requires_grad_(True)
    y64 = plain(x64, m64)
    (y64 * R.f64(w)).sum().backward()
    # the attention's own tolerances: bf16 Q, K, V and O inside
    assert rel_l2(to_np(y), y64.detach().numpy()) <= O_REL_L2
    assert rel_l2(to_np(x.grad), x64.grad.numpy()) <= GRAD_REL_L2
    assert rel_l2(to_np(modulation.grad), m64.grad.numpy()) <= GRAD_REL_L2
    for block, ref in zip(stack.blocks, plain.blocks):
        for name, p in block.named_parameters():
            assert rel_l2(to_np(p.grad), ref[name].grad.numpy()) <= GRAD_REL_L2, name
    # one block after the other, without the joined passes: the same bits
    z = x.detach()
    for i, block in enumerate(stack.blocks):
        z = block(z, grid.to(DEV), modulation.detach()[:, :, i])
    assert torch.equal(z, y.detach())


def test_blocks_without_positions_or_modulation():
    gen = torch.Generator().manual_seed(7)
    x = _rand(gen, 1, 130, 64)
    plain = train.AttentionBlock(64, 1, 64, generator=torch.Generator().manual_seed(1))
    normed = train.AttentionBlock(64, 1, 64, generator=torch.Generator().manual_seed(1),
                                  norm="layer")
    want = x + plain(train.residual_norm(x)[1])
    got = normed(x)
    assert (got - want).abs().max() <= 2.0 ** -23 * want.abs().max()  # a sum, rounded once each
    with pytest.raises(ValueError):
        plain(x, modulation=torch.zeros(1, 1, 3, 64, device=DEV))
    with pytest.raises(ValueError):
        train.BlockStack([plain])


def test_distillation_step_clips():
    c, h, d, n = 64, 1, 64, 130
    teacher, student = _stack(c, h, d, 8), _stack(c, h, d, 9)
    for p in teacher.parameters():
        p.requires_grad_(False)
    g = torch.Generator().manual_seed(10)
    x = _rand(g, 1, n, c)
    inputs = dict(grid=torch.tensor([[2, 5, 13]], dtype=torch.int32, device=DEV),
                  modulation=_rand(g, 1, 1, 2, 3, c, std=0.3))
    before = [p.detach().double().clone() for p in student.parameters()]
    opt = torch.optim.SGD(student.parameters(), lr=1.0)
    loss = train.distillation_step(student, teacher, x, opt, max_grad_norm=1e-3, **inputs)
    assert loss > 0
    grads = torch.stack([p.grad.double().norm() for p in student.parameters()]).norm()
    # norm / (norm + eps) of the bound, with a rounding of each gradient
    assert 1e-3 * (1 - 1e-4) <= float(grads) <= 1e-3 * (1 + 2.0 ** -20)
    for p, q in zip(student.parameters(), before):
        step = (p.detach().double() - q).norm()
        assert float((step - p.grad.double().norm()).abs()) <= 2.0 ** -24 * float(q.norm()) + 1e-9
    norm = train.clip_grad_norm_(student.parameters(), 1.0)
    assert float(norm) == pytest.approx(float(grads), rel=2.0 ** -18)
    for p in student.parameters():
        p.grad = None
    assert float(train.clip_grad_norm_(student.parameters(), 1.0)) == 0.0
    before = [p.detach().clone() for p in student.parameters()]
    plain = train.distillation_step(student, teacher, x, opt, **inputs)
    assert plain > 0 and any(not torch.equal(p, q) for p, q in zip(student.parameters(), before))


def test_forward_and_backward_captured_into_a_graph():
    g = torch.Generator().manual_seed(11)
    x, br = _rand(g, 2, 50, 256, grad=True), _rand(g, 2, 50, 256, grad=True)
    table = _rand(g, 2, 1, 3, 256, grad=True)
    w = _rand(g, 256, mean=1.0, grad=True)
    dq = _rand(g, 2, 2, 50, 128, dtype=BF)
    leaves = (x, br, table, w)

    def step():
        y, h = train.residual_norm(x, br, table[:, :, 2], table[:, :, 1], table[:, :, 0])
        q = train.qkv_heads(h.unflatten(-1, (2, 128)), norm="token", q_weight=w)[0]
        return y, torch.autograd.grad([q, y], leaves, [dq, y.detach()])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, grads = step()
    with torch.no_grad():
        for t in leaves:
            t.mul_(0.75)
    graph.replay()
    torch.cuda.synchronize()
    y2, want = step()
    assert torch.equal(y, y2)
    for a, b in zip(grads, want):
        assert torch.equal(a, b)
