"""Orthogonalised updates (sparge_orthogonalize, sparge_muon_step) against 64 bits."""

import math

import pytest
import torch

from block_sparse_attention_sparge_gb300 import binding as B
from ortho_reference import ROUND, check, reference

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def _rand(seed, *shape, dtype=F32, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


SHAPES = [
    [(1, 1)], [(1, 77)], [(77, 1)], [(2, 2)], [(128, 128)], [(127, 129)], [(129, 127)],
    [(64, 1001)], [(1001, 64)], [(256, 384)], [(300, 300)], [(700, 333)], [(16, 5000)],
    [(1536, 24)], [(640, 1536)], [(1153, 1000)],
    [(128, 128)] * 4, [(5, 9), (400, 130), (130, 400), (1, 1), (257, 256)],
    [(33, 65)] * 65,                      # more than one batch
]


@pytest.mark.parametrize("k", range(len(SHAPES)))
@pytest.mark.parametrize("dtype", [BF, F32])
def test_lists(k, dtype):
    gs = [_rand(100 * k + i, *s, dtype=dtype, std=1e-3) for i, s in enumerate(SHAPES[k])]
    keep = [g.clone() for g in gs]
    outs = B.sparge_orthogonalize(gs, check_status=True)
    for g, o, b in zip(gs, outs, keep):
        assert o.dtype == dtype and torch.equal(g, b)
        check(o, reference(g), dtype == BF)
    again = B.sparge_orthogonalize(gs)
    for a, o in zip(again, outs):
        assert torch.equal(a, o)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_either_form_for_either_type(half, dtype):
    g = _rand(1, 200, 300, dtype=dtype)
    check(B.sparge_orthogonalize([g], half=half)[0], reference(g), half)


def test_mixed_types_in_one_list():
    gs = [_rand(i, 140, 90 + i, dtype=t) for i, t in enumerate((BF, F32, F32, BF))]
    for g, o in zip(gs, B.sparge_orthogonalize(gs)):
        assert o.dtype == g.dtype
        check(o, reference(g), g.dtype == BF)


def test_a_few_strong_directions():
    """The usual gradient: the products' rounding is not amplified with the weak ones."""
    g = _rand(2, 500, 8) @ _rand(3, 8, 700) + 0.02 * _rand(4, 500, 700)
    check(B.sparge_orthogonalize([g], half=True)[0], reference(g), True)
    check(B.sparge_orthogonalize([g])[0], reference(g), False, scale=4.0)


@pytest.mark.parametrize("steps,coefficients", [(0, (1.0, 0.0, 0.0)), (1, (1.5, -0.5, 0.0)),
                                                (3, (1.875, -1.25, 0.375)), (10, (1.5, -0.5, 0.0))])
def test_steps_and_coefficients(steps, coefficients):
    for shape in ((150, 260), (260, 150)):
        g = _rand(5, *shape)
        o = B.sparge_orthogonalize([g], steps=steps, coefficients=coefficients)[0]
        check(o, reference(g, steps, coefficients), False)


@pytest.mark.parametrize("size", [1e-37, 1e-30, 1e-12, 1e12, 1e30, 1e37])
def test_sizes_whose_squares_leave_fp32(size):
    g = _rand(6, 130, 200) * size
    o = B.sparge_orthogonalize([g], eps=0.0)[0]
    check(o, reference(g, eps=0.0), False)


def test_eps_zeros_infinities_and_nan():
    z = torch.zeros(130, 70, device=DEV)
    one = _rand(7, 130, 70)
    bad, inf = one.clone(), one.clone()
    bad[3, 4] = float("nan")
    inf[100, 69] = float("inf")
    out = B.sparge_orthogonalize([z, one, bad, inf, one.bfloat16()])
    assert (out[0] == 0).all() and out[2].isnan().all() and out[3].isnan().all()
    check(out[1], reference(one), False)
    check(out[4], reference(one.bfloat16()), True)
    tiny = one * 1e-9
    check(B.sparge_orthogonalize([tiny], eps=1e-6)[0], reference(tiny, eps=1e-6), False)


def test_rows_and_columns_of_any_stride_and_their_surroundings():
    buf = _rand(8, 300, 1000)
    for view in (buf[:, 3:204], buf[5:130, 8:520], buf.t()[:200, :150], buf[::2, :77],
                 buf.t()[7:300, 1:100]):
        o = B.sparge_orthogonalize([view])[0]
        assert o.shape == view.shape
        check(o, reference(view), False)
        wide = torch.full((1100, 1100), 9.0, device=DEV)
        into = (wide.t() if view.stride(0) == 1 else wide)[10:10 + view.shape[0], 3:3 + view.shape[1]]
        version = wide._version
        B.sparge_orthogonalize([view], out=[into])
        assert torch.equal(into, o) and wide._version > version
        into.fill_(9.0)
        assert (wide == 9).all()
    # in its own place
    own = buf[:200, 100:260].clone()
    want = B.sparge_orthogonalize([own])[0]
    B.sparge_orthogonalize([own], out=[own])
    assert torch.equal(own, want)


@pytest.mark.parametrize("wtype,gtype", [(F32, F32), (BF, BF), (F32, BF)])
@pytest.mark.parametrize("nesterov", [True, False])
def test_step(wtype, gtype, nesterov):
    shapes = [(128, 128), (300, 140), (140, 300), (1, 50)]
    lr, mu, wd = 0.1, 0.9, 0.3
    ws = [_rand(i, *s, dtype=wtype, std=0.1) for i, s in enumerate(shapes)]
    ms = [_rand(10 + i, *s, std=0.5) for i, s in enumerate(shapes)]
    for rms in (None, 0.2):
        gs = [_rand(20 + i, *s, dtype=gtype) for i, s in enumerate(shapes)]
        w0, m0 = [w.double() for w in ws], [m.double() for m in ms]
        versions = [t._version for t in ws + ms]
        B.sparge_muon_step(ws, gs, ms, lr, momentum=mu, nesterov=nesterov, weight_decay=wd, rms=rms,
                           check_status=True)
        assert all(t._version > v for t, v in zip(ws + ms, versions))
        for w, g, m, a, b in zip(ws, gs, ms, w0, m0):
            want_m = mu * b + g.double()
            # (mu as fp32, one product and one sum)
            assert ((m.double() - want_m).abs() <= 3 * 2.0 ** -24 * (mu * b.abs() + g.double().abs())).all()
            u = g.double() + mu * want_m if nesterov else want_m
            r, c = w.shape
            gain = math.sqrt(max(1, r / c)) if rms is None else rms * math.sqrt(max(r, c))
            o = lr * gain * reference(u)
            want = (1 - lr * wd) * a - o
            assert w.dtype == wtype
            # (keep and step as fp32)
            off = (w.double() - want).norm() - 2.0 ** -23 * (a.norm() + o.norm())
            assert off <= ROUND[wtype] * want.norm() + (2.0 ** -8.5 if wtype == BF else 2.0 ** -17) * o.norm()


def test_step_without_momentum():
    w, g = _rand(1, 90, 60), _rand(2, 90, 60)
    want = w.double() - 0.5 * math.sqrt(1.5) * reference(g)
    B.sparge_muon_step([w], [g], None, 0.5)
    check(w, want, False)


def test_captured_replayed_and_on_two_streams():
    gs = [_rand(1, 200, 100), _rand(2, 64, 300, dtype=BF)]
    outs = [torch.empty_like(g) for g in gs]
    B.sparge_orthogonalize(gs, out=outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.sparge_orthogonalize(gs, out=outs)
    for seed in (5, 6):
        for g in gs:
            g.copy_(_rand(seed, *g.shape, dtype=g.dtype))
        graph.replay()
        torch.cuda.synchronize()
        for g, o in zip(gs, outs):
            check(o, reference(g), g.dtype == BF)
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for _ in range(3):
        for s, g in zip(streams, gs):
            with torch.cuda.stream(s):
                got.append((g, B.sparge_orthogonalize([g])[0]))
    torch.cuda.synchronize()
    for g, o in got:
        check(o, reference(g), g.dtype == BF)


def test_a_large_matrix_and_a_long_list():
    g = _rand(1, 2304, 4736, dtype=BF)
    check(B.sparge_orthogonalize([g])[0], reference(g), True)
    gs = [_rand(i, 100 + i % 90, 150, dtype=BF) for i in range(200)]
    for g, o in zip(gs, B.sparge_orthogonalize(gs)):
        check(o, reference(g), True)


def test_refusals_on_the_device():
    a, b = _rand(1, 20, 30), _rand(2, 20, 30)
    for bad in ([], [a[0]], [a.half()], [a, b.cpu()], [a[:, ::2]]):
        with pytest.raises(ValueError):
            B.sparge_orthogonalize(bad)
    for out in ([], [a.t()], [a.half()], [torch.empty(30, 20, device=DEV).t()]):
        with pytest.raises(ValueError):
            B.sparge_orthogonalize([a], out=out)
    with pytest.raises(ValueError):
        B.sparge_muon_step([a], [b], [a.bfloat16()], 0.1)
    with pytest.raises(ValueError):
        B.sparge_muon_step([a], [b, b], None, 0.1)
    big = _rand(3, 60, 100)
    for mats, kw in (([a, b], dict(out=[a, a])), ([a], dict(out=[a[:0].new_empty(1).expand(20, 30)])),
                     ([big[:20, :30]], dict(out=[big[:20, 1:31]])),
                     ([big[:20, :30], b], dict(out=[a, big[10:30, 20:50]])),
                     ([a], dict(coefficients=(float("nan"), 1, 1))), ([a], dict(steps=-1)),
                     ([a], dict(eps=float("inf"))),
                     ([a], dict(workspace=torch.empty(64, dtype=torch.uint8, device=DEV)))):
        with pytest.raises((B.SpargeError, ValueError)):
            B.sparge_orthogonalize(mats, **kw)
    with pytest.raises(B.SpargeError):
        B.sparge_muon_step([a], [a], None, 0.1)       # the gradient is the weight
    with pytest.raises(B.SpargeError):
        B.sparge_muon_step([a], [b], [a], 0.1)
    with pytest.raises(B.SpargeError):
        B.sparge_muon_step([a, a], [b, b], None, 0.1)
    # columns of one buffer lie beside one another
    B.sparge_orthogonalize([big[:, :40], big[:, 40:90]], out=[big[:, :40], big[:, 40:90]])
