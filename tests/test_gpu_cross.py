"""Attention over a context (sparge_cross_fwd / _bwd) against 64 bits."""

import pytest
import torch

from block_sparse_attention_sparge_gb300 import binding as B
from cross_reference import check, reference

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _make(shape, seed=0, layout="heads", garbage=None, lens=None):
    """q, k, v, dout of (B, Bk, H, Hk, N, M, d); ``garbage``: what stands behind the lengths."""
    b, bk, h, hk, n, m, d = shape
    g = torch.Generator().manual_seed(seed)

    def rand(bb, hh, nn):
        if layout == "tokens":
            return torch.randn((bb, nn, hh, d), generator=g).to(BF).to(DEV).transpose(1, 2)
        return torch.randn((bb, hh, nn, d), generator=g).to(BF).to(DEV)

    q, k, v, do = rand(b, h, n), rand(bk, hk, m), rand(bk, hk, m), rand(b, h, n)
    if layout == "fused":  # key and value as slices of one projection, values last
        kv = torch.cat([k.transpose(1, 2), v.transpose(1, 2)], 2)  # [bk, m, 2 hk, d]
        k, v = kv[:, :, :hk].transpose(1, 2), kv[:, :, hk:].transpose(1, 2)
    if garbage is not None:
        for t in (k, v):
            for i in range(bk):
                used = max(lens) if bk == 1 else lens[i]
                t[i, :, max(0, used):] = garbage
    return q, k, v, do


def _lens(lens):
    return None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)


CASES = [
    ((1, 1, 2, 2, 100, 33, 64), None),
    ((1, 1, 1, 1, 1, 1, 128), None),
    ((1, 1, 1, 1, 1, 2, 64), None),
    ((1, 1, 3, 3, 130, 1, 64), None),
    ((2, 2, 4, 2, 129, 257, 64), [257, 100]),
    ((2, 2, 4, 1, 128, 128, 128), [128, 64]),
    ((3, 3, 3, 3, 65, 200, 128), [0, 200, 1]),
    ((3, 1, 6, 3, 200, 130, 128), [130, 129, 5]),
    ((4, 1, 2, 1, 77, 300, 64), [300, 0, 128, 129]),
    ((2, 1, 2, 2, 256, 64, 128), None),
    ((5, 5, 2, 2, 3, 70, 64), [70, 63, 64, 65, -3]),
    ((2, 2, 2, 2, 1000, 512, 128), [512, 999]),     # a length beyond the context
    ((1, 1, 12, 12, 2500, 512, 128), None),         # several parts of the query tiles
    ((1, 1, 5, 5, 1537, 385, 64), None),
    ((2, 2, 2, 1, 1, 5000, 128), [5000, 4321]),     # parts of the keys
    ((1, 1, 1, 1, 64, 9000, 64), None),
    ((3, 1, 1, 1, 7, 3001, 128), [3001, 0, 260]),
    ((1, 1, 1, 1, 20000, 40, 64), None),
    # query tiles that fill the machine
    ((40, 40, 4, 4, 129, 66, 64), None),
    ((1, 1, 12, 12, 3500, 512, 128), None),
    ((3, 3, 12, 3, 1200, 300, 128), [300, 0, 129]),
    ((7, 1, 6, 2, 1000, 400, 64), [400, 1, 0, 128, 257, 399, 3]),
    ((80, 80, 4, 2, 1, 200, 64), None),
    ((80, 80, 5, 1, 2, 129, 128), [129 - (i * 7) % 130 for i in range(80)]),
    ((1, 1, 3, 3, 13100, 700, 64), None),
    ((311, 1, 1, 1, 100, 130, 128), None),
]


@pytest.mark.parametrize("k", range(len(CASES)))
@pytest.mark.parametrize("layout", ["heads", "tokens", "fused"])
def test_forward(k, layout):
    shape, lens = CASES[k]
    q, kk, v, _ = _make(shape, k, layout)
    o, lse = B.sparge_cross_fwd(q, kk, v, _lens(lens), check_status=True)
    out, lim = reference(q, kk, v, lens)
    check((o, lse), out, lim, ("o", "lse"))


@pytest.mark.parametrize("k", range(len(CASES)))
@pytest.mark.parametrize("layout", ["heads", "tokens"])
def test_backward(k, layout):
    shape, lens = CASES[k]
    q, kk, v, do = _make(shape, k, layout)
    ln = _lens(lens)
    o, lse = B.sparge_cross_fwd(q, kk, v, ln)
    got = B.sparge_cross_bwd(q, kk, v, o, lse, do, ln, check_status=True)
    out, lim = reference(q, kk, v, lens, dout=do)
    check(got, out, lim, ("dq", "dk", "dv"))
    again = B.sparge_cross_bwd(q, kk, v, o, lse, do, ln)
    for a, b in zip(got, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("garbage", [float("nan"), float("inf"), -3.3e38])
@pytest.mark.parametrize("k", [4, 5, 6, 7, 8, 10, 14, 16, 20, 21, 23])
def test_what_lies_behind_the_lengths_is_not_used(k, garbage):
    shape, lens = CASES[k]
    q, kk, v, do = _make(shape, k, "tokens", garbage, lens)
    clean = _make(shape, k, "tokens", 0.0, lens)
    ln = _lens(lens)
    o, lse = B.sparge_cross_fwd(q, kk, v, ln)
    ref = B.sparge_cross_fwd(*clean[:3], ln)
    assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
    got = B.sparge_cross_bwd(q, kk, v, o, lse, do, ln)
    for a, b in zip(got, B.sparge_cross_bwd(*clean[:3], o, lse, do, ln)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("scale", [0.02, -0.1, 1.0])
def test_scales(scale):
    shape, lens = CASES[4]
    q, k, v, do = _make(shape, 3)
    if scale == 1.0:
        q = q * 0.25
    ln = _lens(lens)
    o, lse = B.sparge_cross_fwd(q, k, v, ln, softmax_scale=scale)
    out, lim = reference(q, k, v, lens, scale, do)
    check((o, lse), out, lim, ("o", "lse"))
    check(B.sparge_cross_bwd(q, k, v, o, lse, do, ln, softmax_scale=scale), out, lim,
          ("dq", "dk", "dv"))


@pytest.mark.parametrize("batch", [1, 80])
@pytest.mark.parametrize("d", [64, 128])
def test_logits_that_grow_from_step_to_step(batch, d):
    """The running maximum moves by more than the kernel's bound for rescaling, both
    ways, and a last key outweighs all before."""
    q, k, v, _ = _make((batch, 1, 2, 2, 140, 700, d), 5)
    ramp = torch.linspace(-3, 3, 700, device=DEV)
    k = k * 0.1 + (ramp[:, None] * torch.ones(d, device=DEV)).to(BF)
    q = (q * 0.1 + 1.0).to(BF)
    q[:, :, ::2] *= -1
    for lens in (None, [651] * batch):
        o, lse = B.sparge_cross_fwd(q, k, v, _lens(lens))
        out, lim = reference(q, k, v, lens)
        check((o, lse), out, lim, ("o", "lse"))


def test_given_outputs_and_their_surroundings():
    shape, lens = CASES[7]
    b, bk, h, hk, n, m, d = shape
    q, k, v, do = _make(shape, 7)
    ln = _lens(lens)
    ref = B.sparge_cross_fwd(q, k, v, ln)
    wide = torch.full((b, n, 2 * h, d), 7.0, dtype=BF, device=DEV)
    o = wide[:, :, :h].transpose(1, 2)
    lse = torch.empty(b, h, n, device=DEV)
    before = wide._version
    got = B.sparge_cross_fwd(q, k, v, ln, out=o, lse=lse)
    assert got[0] is o and got[1] is lse and wide._version > before
    assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1]) and (wide[:, :, h:] == 7).all()
    # gradients of a fused key-value projection, side by side in one buffer
    want = B.sparge_cross_bwd(q, k, v, *ref, do, ln)
    dkv = torch.full((bk, m, 3, hk, d), 7.0, dtype=BF, device=DEV)
    dq = torch.empty(b, n, h, d, dtype=BF, device=DEV).transpose(1, 2)
    outs = (dq, dkv[:, :, 0].transpose(1, 2), dkv[:, :, 1].transpose(1, 2))
    B.sparge_cross_bwd(q, k, v, o, lse, do, ln, out=outs)
    for a, w in zip(outs, want):
        assert torch.equal(a, w)
    assert (dkv[:, :, 2] == 7).all()


def test_gradients_against_differences():
    """<gradient, direction> against central differences of the 64-bit forward."""
    shape, lens = (2, 1, 4, 2, 70, 90, 64), [90, 41]
    q, k, v, do = _make(shape, 11)
    ln = _lens(lens)
    o, lse = B.sparge_cross_fwd(q, k, v, ln)
    grads = B.sparge_cross_bwd(q, k, v, o, lse, do, ln)
    out, lim = reference(q, k, v, lens, dout=do)
    ins = [t.double() for t in (q, k, v)]
    g = torch.Generator().manual_seed(1)
    for i, name in enumerate(("dq", "dk", "dv")):
        u = torch.randn(ins[i].shape, generator=g, dtype=torch.float64).to(DEV)
        h, side = 1e-4, []
        for sign in (1, -1):
            moved = [t + sign * h * u if j == i else t for j, t in enumerate(ins)]
            side.append((reference(*moved, lens)[0]["o"] * do.double()).sum())
        want = (side[0] - side[1]) / (2 * h)
        # (h^2 / 6 of the third derivative: below 1e-6 of these sums)
        slack = (lim[name] * u.abs()).sum() + 1e-6 * (out[name] * u).abs().sum()
        assert (grads[i].double() * u).sum().sub(want).abs() <= slack


def test_captured_and_replayed_with_other_lengths():
    shape = (2, 2, 4, 2, 150, 260, 128)
    q, k, v, do = _make(shape, 13)
    ln = _lens([260, 260])
    o, lse = torch.empty_like(q), torch.empty(2, 4, 150, device=DEV)
    outs = [torch.empty_like(t) for t in (q, k, v)]

    def step():
        B.sparge_cross_fwd(q, k, v, ln, out=o, lse=lse)
        B.sparge_cross_bwd(q, k, v, o, lse, do, ln, out=outs)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed, lens in ((14, [130, 0]), (15, [1, 259])):
        for t, new in zip((q, k, v, do), _make(shape, seed)):
            t.copy_(new)
        ln.copy_(_lens(lens))
        graph.replay()
        torch.cuda.synchronize()
        out, lim = reference(q, k, v, lens, dout=do)
        check((o, lse, *outs), out, lim, ("o", "lse", "dq", "dk", "dv"))


def test_streams_run_beside_one_another():
    """Calls on two streams have workspaces of their own."""
    runs = []
    for i in range(2):
        q, k, v, do = _make((1, 1, 2, 2, 700, 300, 64), 20 + i)
        runs.append((torch.cuda.Stream(), q, k, v, do))
    torch.cuda.synchronize()
    got = []
    for s, q, k, v, do in runs * 3:
        with torch.cuda.stream(s):
            o, lse = B.sparge_cross_fwd(q, k, v)
            got.append(B.sparge_cross_bwd(q, k, v, o, lse, do))
    torch.cuda.synchronize()
    for i, (_, q, k, v, do) in enumerate(runs):
        out, lim = reference(q, k, v, dout=do)
        for j in range(i, 6, 2):
            check(got[j], out, lim, ("dq", "dk", "dv"))


def test_a_context_whose_offsets_pass_32_bits():
    """Keys of 20 heads of 131072 tokens in token-major order: the last token lies
    2^31 elements and more behind the first."""
    h, m, d = 132, 131072, 128
    kv = torch.zeros(1, m, h, d, dtype=BF, device=DEV)
    g = torch.Generator().manual_seed(2)
    n = 3
    q = torch.randn((1, h, n, d), generator=g).to(BF).to(DEV)
    kv[:, -200:] = torch.randn((1, 200, h, d), generator=g).to(BF).to(DEV)
    k = kv.transpose(1, 2)
    o, lse = B.sparge_cross_fwd(q, k, k)
    for head in (0, h - 1):
        out, lim = reference(q[:, head:head + 1], k[:, head:head + 1], k[:, head:head + 1])
        check((o[:, head:head + 1], lse[:, head:head + 1]), out, lim, ("o", "lse"))


def test_refusals_on_the_device():
    q, k, v, do = _make((2, 2, 4, 2, 20, 30, 64), 1)
    o, lse = B.sparge_cross_fwd(q, k, v)
    ln = _lens([3, 4])
    for bad in ((q.float(), k, v), (q, k[:, :, :, :32], v), (q, k, v[:, :, :20]), (q, k, v.cpu()),
                (q.transpose(2, 3), k, v), (q[0], k, v)):
        with pytest.raises(ValueError):
            B.sparge_cross_fwd(*bad)
    for bad in (ln.long(), ln[:1], ln.cpu()):
        with pytest.raises(ValueError):
            B.sparge_cross_fwd(q, k, v, bad)
    for kw in (dict(out=o[:, :2]), dict(out=o.float()), dict(lse=lse[:1]), dict(lse=lse.double())):
        with pytest.raises(ValueError):
            B.sparge_cross_fwd(q, k, v, **kw)
    three = _make((2, 2, 4, 3, 20, 30, 64), 1)
    odd = torch.zeros(2 * 4 * 20 * 64 + 8, dtype=BF, device=DEV)[1:-7].view(2, 4, 20, 64)
    wide = torch.zeros(2, 4, 20, 68, dtype=BF, device=DEV)[..., :64]
    for args, kw, code in (((three[0], *three[1:3]), {}, B.SPARGE_ERR_INVALID_ARG),
                           ((q, k[:, :, :, :].expand(2, 2, 30, 64)[:, :1].expand(2, 2, 30, 64), v),
                            {}, B.SPARGE_ERR_INVALID_ARG),
                           ((odd, k, v), {}, B.SPARGE_ERR_MISALIGNED),
                           ((wide, k, v), {}, B.SPARGE_ERR_MISALIGNED),
                           ((q, k, v), dict(out=q), B.SPARGE_ERR_INVALID_ARG),
                           ((q, k, v), dict(softmax_scale=float("nan")), B.SPARGE_ERR_INVALID_ARG),
                           ((_make((3, 2, 4, 2, 20, 30, 64))[:3]), {}, B.SPARGE_ERR_INVALID_ARG),
                           ((q.new_zeros(2, 4, 20, 80), k.new_zeros(2, 2, 30, 80),
                             k.new_zeros(2, 2, 30, 80)), {}, B.SPARGE_ERR_UNSUPPORTED)):
        with pytest.raises(B.SpargeError) as e:
            B.sparge_cross_fwd(*args, **kw)
        assert e.value.code == code, (args[0].shape, kw)
    for kw in (dict(out=(q, k, v)), dict(out=(torch.empty_like(q), torch.empty_like(k)) + (q[:, :2, :, :],)),
               dict(workspace=torch.empty(64, dtype=torch.uint8, device=DEV))):
        with pytest.raises((B.SpargeError, ValueError)):
            B.sparge_cross_bwd(q, k, v, o, lse, do, **kw)
    same = torch.empty_like(k)
    with pytest.raises(B.SpargeError):
        B.sparge_cross_bwd(q, k, v, o, lse, do, out=(torch.empty_like(q), same, same))
