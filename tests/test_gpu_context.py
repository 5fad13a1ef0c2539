"""Blocks that attend to a context, and their training: gradients of the whole stack
against a 64-bit model of it, the optimiser's step on them, and both captured."""

import math

import pytest
import torch

from block_sparse_attention_sparge_gb300 import train
from ortho_reference import ROUND, reference as orthogonal

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
EPS = 1e-6
# A gradient of the stack passes at most some twelve roundings to bf16 (q, k, v, P, O and
# dO, dS, dQ, dK, dV of a block, twice), 2^-8 / sqrt(3) each in the mean square, independent
# of one another: sqrt(12) * 2^-8.8 = 2^-7; twice that for those that are amplified by a
# softmax's or a norm's cancellation.
OFF = 2.0 ** -6


def _rand(seed, *shape, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(DEV)


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _norm(x, kind):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    return x / (x.square().mean(-1, keepdim=True) + EPS).sqrt()


def _rms(x, w, kind):
    dims = (2, 3) if kind == "token" else (3,)
    w = w.view(x.shape[2:] if kind == "token" else (x.shape[3],))
    return x / (x.square().mean(dims, keepdim=True) + EPS).sqrt() * w


def _attend(block, w, h, context, kv_len):
    """A block's attention in 64 bits (dense, without positions)."""
    cross = isinstance(block, train.CrossAttentionBlock)
    src = context if cross else h
    q = (h @ w["wq"]).unflatten(-1, (block.heads, -1))
    hk = block.kv_heads if cross else block.heads
    k, v = ((src @ w[n]).unflatten(-1, (hk, -1)) for n in ("wk", "wv"))
    if block.qk_norm is not None:
        q, k = _rms(q, w["norm_q"], block.qk_norm), _rms(k, w["norm_k"], block.qk_norm)
    q, k, v = (t.transpose(1, 2) for t in (q, k, v))
    k, v = (t.repeat_interleave(block.heads // hk, 1) for t in (k, v))
    s = q @ k.transpose(-1, -2) / math.sqrt(block.head_dim)
    if cross and kv_len is not None:
        s = s.masked_fill(torch.arange(s.shape[-1], device=DEV) >= kv_len[:, None, None, None],
                          -math.inf)
    p = torch.where((s > -math.inf).any(-1, keepdim=True), s.softmax(-1), 0.0).nan_to_num(0.0)
    return (p @ v).transpose(1, 2).flatten(2) @ w["wo"]


def _model(blocks, weights, x, context, kv_len):
    for block, w in zip(blocks, weights):
        x = x + _attend(block, w, _norm(x, block.norm), context, kv_len)
    return x


def _weights(blocks):
    return [{n: p.detach().double().requires_grad_(True) for n, p in b.named_parameters()}
            for b in blocks]


def _stack(qk_norm=None, seed=1):
    return [train.AttentionBlock(128, 2, 64, generator=_gen(seed), qk_norm=qk_norm, norm="layer"),
            train.CrossAttentionBlock(128, 4, 64, 96, kv_heads=2, generator=_gen(seed + 1),
                                      qk_norm=qk_norm, norm="rms"),
            train.AttentionBlock(128, 2, 64, generator=_gen(seed + 2), norm="layer"),
            train.CrossAttentionBlock(128, 2, 64, 96, generator=_gen(seed + 3), norm="layer")]


@pytest.mark.parametrize("qk_norm", [None, "token", "head"])
@pytest.mark.parametrize("shared", [False, True])
def test_gradients_of_a_stack(qk_norm, shared):
    blocks = _stack(qk_norm)
    stack = train.BlockStack(blocks)
    x = _rand(5, 2, 200, 128).requires_grad_(True)
    context = _rand(6, 1 if shared else 2, 90, 96).requires_grad_(True)
    kv_len = torch.tensor([90, 31], dtype=torch.int32, device=DEV)
    up = _rand(7, 2, 200, 128)
    y = stack(x, context=context, kv_len=kv_len)
    (y * up).sum().backward()
    weights = _weights(blocks)
    x64, c64 = (t.detach().double().requires_grad_(True) for t in (x, context))
    want = _model(blocks, weights, x64, c64, kv_len)
    (want * up.double()).sum().backward()
    assert (y.double() - want).norm() <= OFF * want.norm()
    pairs = [("x", x.grad, x64.grad), ("context", context.grad, c64.grad)]
    for i, (b, w) in enumerate(zip(blocks, weights)):
        pairs += [(f"{i}.{n}", p.grad, w[n].grad) for n, p in b.named_parameters()]
    for name, got, ref in pairs:
        assert got.shape == ref.shape and got.dtype == torch.float32
        assert (got.double() - ref).norm() <= OFF * ref.norm(), name


def test_cross_attention_of_any_views():
    """A fused projection's slices, an expanded gradient, a sample without context."""
    kv = _rand(1, 3, 70, 2, 2, 64).to(BF).requires_grad_(True)
    q = _rand(2, 3, 50, 4, 64).to(BF).requires_grad_(True)
    kv_len = torch.tensor([70, 0, 12], dtype=torch.int32, device=DEV)
    o = train.cross_attention(q.transpose(1, 2), kv[:, :, 0].transpose(1, 2),
                              kv[:, :, 1].transpose(1, 2), kv_len)
    assert o.transpose(1, 2).is_contiguous()
    o.sum().backward()
    q64, kv64 = (t.detach().double().requires_grad_(True) for t in (q, kv))
    k64, v64 = (kv64[:, :, i].transpose(1, 2).repeat_interleave(2, 1) for i in range(2))
    s = q64.transpose(1, 2) @ k64.transpose(-1, -2) / 8
    s = s.masked_fill(torch.arange(70, device=DEV) >= kv_len[:, None, None, None], -1e30)
    p = s.softmax(-1) * (kv_len > 0)[:, None, None, None]
    (p @ v64).sum().backward()
    assert (o[1] == 0).all() and (q.grad[1] == 0).all() and (kv.grad[1] == 0).all()
    for got, ref in ((q.grad, q64.grad), (kv.grad, kv64.grad)):
        assert (got.double() - ref).norm() <= OFF * ref.norm()


def test_a_training_step():
    """distillation_step with the cross attention and Muon: every weight moves by the
    orthogonalised gradient of that step."""
    stack = train.BlockStack(_stack("head"))
    teacher = train.BlockStack(_stack("head", seed=30))
    teacher.requires_grad_(False)
    mats = [p for p in stack.parameters() if p.dim() == 2]
    rest = [p for p in stack.parameters() if p.dim() != 2]
    muon = train.Muon(mats, lr=0.03, momentum=0.9, weight_decay=0.1)
    inputs = dict(context=_rand(3, 2, 60, 96),
                  kv_len=torch.tensor([60, 20], dtype=torch.int32, device=DEV))
    x = _rand(4, 2, 150, 128)
    m = [torch.zeros_like(p, dtype=torch.float64) for p in mats]
    for _ in range(3):
        before = [p.detach().double().clone() for p in mats]
        kept = [p.detach().clone() for p in rest]
        loss = train.distillation_step(stack, teacher, x, muon, max_grad_norm=1.0, **inputs)
        assert math.isfinite(loss)
        for i, (p, b) in enumerate(zip(mats, before)):
            m[i] = 0.9 * m[i] + p.grad.double()
            gain = math.sqrt(max(1, p.shape[0] / p.shape[1]))
            step = 0.03 * gain * orthogonal(p.grad.double() + 0.9 * m[i])
            want = (1 - 0.03 * 0.1) * b - step
            off = 2.0 ** -8.5 * step.norm() + (ROUND[p.dtype] + 2.0 ** -23) * want.norm()
            assert (p.detach().double() - want).norm() <= off
            # (a momentum's roundings to fp32)
            assert (muon.state[p]["momentum"].double() - m[i]).norm() <= 2.0 ** -21 * m[i].norm()
        for p, k in zip(rest, kept):
            assert torch.equal(p, k)


def test_optimiser_state_survives_a_checkpoint():
    w = [torch.nn.Parameter(_rand(i, 40, 30 + i).to(BF)) for i in range(2)]
    opt = train.Muon(w, lr=0.1)
    for p in w:
        p.grad = _rand(9, *p.shape).to(BF)
    opt.step()
    copies = [torch.nn.Parameter(p.detach().clone()) for p in w]
    other = train.Muon(copies, lr=0.5)
    other.load_state_dict(opt.state_dict())
    for p, c in zip(w, copies):
        c.grad = p.grad.clone()
        assert torch.equal(opt.state[p]["momentum"], other.state[c]["momentum"])
        assert other.state[c]["momentum"].dtype == torch.float32
    opt.step()
    other.step()
    for p, c in zip(w, copies):
        assert torch.equal(p, c)


def test_muon_takes_gradients_of_another_order_and_skips_missing_ones():
    a, b, c = (torch.nn.Parameter(_rand(i, 50, 70)) for i in range(3))
    t = torch.nn.Parameter(_rand(5, 70, 50).t())
    g = _rand(7, 50, 70)
    a.grad, t.grad = g.t().contiguous().t(), g.clone()
    before = [p.detach().clone() for p in (a, b, t)]
    opt = train.Muon([a, b, t], lr=0.1, half=None)
    assert opt.step(lambda: 3.0) == 3.0
    assert torch.equal(b, before[1])
    for p, w in ((a, before[0]), (t, before[2])):
        want = w.double() - 0.1 * orthogonal(g.double() * 1.95)
        assert (p.detach().double() - want).norm() <= 2.0 ** -17 * 0.1 * 50 ** 0.5 + 2.0 ** -23 * want.norm()
    with pytest.raises(ValueError):
        train.Muon([torch.nn.Parameter(_rand(1, 5))])


def test_captured_step_beside_a_living_eager_graph():
    """Forward, backward and the optimiser's step captured and replayed while an eager
    graph of the same leaves, of the captured stream, is alive.  (One of another
    stream makes torch wait for that stream, which no capture allows.)"""
    blocks = [train.CrossAttentionBlock(64, 1, 64, 64, generator=_gen(3), norm="rms")]
    stack = train.BlockStack(blocks)
    opt = train.Muon(list(stack.parameters()), lr=0.01)
    x, context = _rand(1, 1, 40, 64), _rand(2, 1, 30, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager = stack(x, context=context)
        grads = torch.autograd.grad(stack(x, context=context).square().sum(), list(stack.parameters()))
        for p, g in zip(stack.parameters(), grads):
            p.grad = g.clone()
        opt.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        loss = stack(x, context=context).square().sum()
        for p, g in zip(stack.parameters(), torch.autograd.grad(loss, list(stack.parameters()))):
            p.grad.copy_(g)
        opt.step()
    torch.cuda.current_stream().wait_stream(side)
    before = [p.detach().clone() for p in stack.parameters()]
    momenta = [opt.state[p]["momentum"].clone() for p in stack.parameters()]
    graph.replay()
    torch.cuda.synchronize()
    assert math.isfinite(float(loss))
    for p, b, m in zip(stack.parameters(), before, momenta):
        u = p.grad.double() * 1.95 + 0.95 * 0.95 * m.double()
        step = 0.01 * orthogonal(u)
        want = b.double() - step
        assert (p.detach().double() - want).norm() <= 2.0 ** -8.5 * step.norm() + 2.0 ** -23 * want.norm()
    assert eager.isfinite().all()
