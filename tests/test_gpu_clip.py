"""Gradient norm and clipping (sparge_clip_grads) against 64 bits.

Bounds: sums of squares are fp32 over 64 values and then over four such sums (at
most 16 fused additions, 3 more and 4: 23 * 2^-24 of the sum, half of it after
the root), the rest is fp64; with the rounding of the norm itself 2^-20 in all.  The factor adds its
rounding and a scaled value its own."""

import math

import pytest
import torch

from block_reference import HALF_STEP, f64
from block_sparse_attention_sparge_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def _rand(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


def _norm(ts):
    return math.sqrt(math.fsum(float(f64(t).square().sum()) for t in ts))


def _check(ts, outs, norm, max_norm, eps=1e-6):
    want = _norm(ts)
    assert abs(float(norm) - want) <= 2.0 ** -20 * want
    factor = min(1.0, max_norm / (want + eps))
    for t, o in zip(ts, outs):
        assert o.dtype == t.dtype and o.shape == t.shape
        ref = f64(t) * factor
        off = (f64(o) - ref).abs()
        # 2^-150: half of fp32's smallest step; bf16's is 2^-134
        tiny = 2.0 ** -134 if t.dtype == BF else 2.0 ** -150
        lim = ref.abs() * (HALF_STEP[t.dtype] * (1 + 2.0 ** -18) + 2.0 ** -20 + 2.0 ** -24) + tiny
        assert (off <= lim).all()


LISTS = [
    [((1,), F32)],
    [((128, 128), F32)] * 4,
    [((3, 5), BF), ((1,), BF), ((0,), BF), ((7,), F32), ((0, 4), F32), ((16385,), BF), ((8,), BF)],
    [((1536, 100), BF), ((100,), F32), ((40000,), F32)],
    [((5,), F32)] * 49,
    [((9,), BF)] * 256,
    [((2,), BF)] * 257,
    [((3,), BF), ((11,), F32)] * 600,          # more than one list of 1024
    [((2, 3), F32)] * 2050,
    [(((1 << 24) + 3,), BF), ((1 << 22,), F32)],
]


@pytest.mark.parametrize("k", range(len(LISTS)))
@pytest.mark.parametrize("max_norm", [0.5, 1e9, 0.0])
def test_lists(k, max_norm):
    g = torch.Generator().manual_seed(k)
    ts = [_rand(g, *s, dtype=d) for s, d in LISTS[k]]
    keep = [t.clone() for t in ts]
    outs = [torch.full_like(t, 9.0) for t in ts]
    norm = B.sparge_clip_grads(ts, max_norm, out=outs)
    _check(ts, outs, norm, max_norm)
    for t, o in zip(ts, keep):
        assert torch.equal(t, o)
    assert norm.shape == () and norm.dtype == F32
    alone = B.sparge_clip_grads(ts, None)
    assert torch.equal(alone, norm)
    again = B.sparge_clip_grads(ts, max_norm)  # in place
    assert torch.equal(again, norm)
    for t, o in zip(ts, outs):
        assert torch.equal(t, o)
    if max_norm == 1e9:
        for t, o in zip(ts, keep):
            assert torch.equal(t, o)


def test_views_at_odd_places_and_their_surroundings():
    for dtype in (BF, F32):
        buf = _rand(torch.Generator().manual_seed(1), 70000, dtype=dtype)
        ref = buf.clone()
        cuts = [(1, 20), (21, 21), (23, 16500), (16523, 16524), (16531, 60001)]
        views = [buf[a:b] for a, b in cuts]
        norm = B.sparge_clip_grads(views, 1.0)
        _check([ref[a:b] for a, b in cuts], views, norm, 1.0)
        inside = torch.zeros(70000, dtype=torch.bool, device=DEV)
        for a, b in cuts:
            inside[a:b] = True
        assert torch.equal(buf[~inside], ref[~inside])
        # outputs aligned otherwise than their inputs
        out = torch.zeros_like(buf)
        outs = [out[a + 3:b + 3] for a, b in cuts[2:3]]
        norm = B.sparge_clip_grads([ref[a:b] for a, b in cuts[2:3]], 1.0, out=outs)
        _check([ref[a:b] for a, b in cuts[2:3]], outs, norm, 1.0)
        assert int(torch.count_nonzero(out)) <= cuts[2][1] - cuts[2][0]


def test_dense_tensors_of_another_order():
    g = torch.Generator().manual_seed(2)
    t = _rand(g, 40, 60).t()
    u = _rand(g, 2, 3, 4, 8).permute(0, 3, 1, 2)
    keep = [t.clone(), u.clone()]
    norm = B.sparge_clip_grads([t, u], 1.0)
    _check(keep, [t, u], norm, 1.0)


@pytest.mark.parametrize("size", [1e30, 3e38, 1e-30, 1e-38])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_sizes_whose_squares_leave_fp32(size, dtype):
    g = torch.Generator().manual_seed(3)
    ts = [((torch.rand((n,), generator=g) + 0.1) / 1.1 * size).to(dtype).to(DEV) for n in (5, 20000)]
    ts.append(torch.ones(40, device=DEV) if size < 1 else torch.zeros(40, device=DEV))
    if size < 1:
        ts[2] *= size
    want = _norm(ts)
    outs = [torch.zeros_like(t) for t in ts]
    norm = B.sparge_clip_grads(ts, size, out=outs, eps=0.0)
    if want < 3.4e38:
        _check(ts, outs, norm, size, eps=0.0)
    else:
        # the norm itself is beyond fp32; the factor and the results are not
        assert math.isinf(float(norm))
        for t, o in zip(ts, outs):
            ref = f64(t) * (size / want)
            assert ((f64(o) - ref).abs() <= ref.abs() * (HALF_STEP[t.dtype] + 2.0 ** -19)).all()


def test_mixed_sizes_in_one_thread():
    """Huge and tiny values side by side: the large ones decide."""
    t = torch.full((64,), 1e-20, device=DEV)
    t[::7] = 1e25
    _check([t.clone()], [t], B.sparge_clip_grads([t], 1e24), 1e24)


def test_zeros_infinities_and_nan():
    z = torch.zeros(1000, device=DEV)
    assert float(B.sparge_clip_grads([z], 1.0)) == 0.0 and (z == 0).all()
    a, b = torch.ones(100, device=DEV), torch.ones(100, device=DEV, dtype=BF)
    a[3] = float("inf")
    norm = B.sparge_clip_grads([a, b], 1.0)
    assert math.isinf(float(norm)) and a[3].isnan() and (b == 0).all()
    assert int(torch.count_nonzero(a.nan_to_num(0))) == 0
    a = torch.ones(100, device=DEV)
    a[9] = float("nan")
    b = torch.ones(100, device=DEV, dtype=BF)
    assert math.isnan(float(B.sparge_clip_grads([a, b], 1.0)))
    assert b.isnan().all() and a.isnan().all()
    z = torch.zeros(9, device=DEV)
    assert float(B.sparge_clip_grads([z], 0.0, eps=0.0)) == 0.0 and (z == 0).all()
    e = torch.empty(0, device=DEV)
    assert float(B.sparge_clip_grads([e], 1.0)) == 0.0


def test_captured_replayed_and_repeatable():
    g = torch.Generator().manual_seed(4)
    ts = [_rand(g, 300, 1000, dtype=BF), _rand(g, 77)]
    outs = [torch.empty_like(t) for t in ts]
    B.sparge_clip_grads(ts, 1.0, out=outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = B.sparge_clip_grads(ts, 1.0, out=outs)
    for seed in (5, 6):
        g = torch.Generator().manual_seed(seed)
        for t in ts:
            t.copy_(_rand(g, *t.shape, dtype=t.dtype))
        graph.replay()
        torch.cuda.synchronize()
        _check(ts, outs, norm, 1.0)
        first = [norm.clone(), *[o.clone() for o in outs]]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(first, [norm, *outs]):
            assert torch.equal(a, b)


def test_more_than_2_to_the_31_values():
    n = 2 ** 31 + 9
    t = torch.zeros(n, dtype=BF, device=DEV)
    t[-8:] = 3.0
    t[5] = 4.0
    norm = B.sparge_clip_grads([t], 1.0)
    want = math.sqrt(8 * 9 + 16)
    assert abs(float(norm) - want) <= 2.0 ** -20 * want
    part = t[-9:].cpu().double()
    assert part[0] == 0
    assert (part[1:] - 3 / want).abs().max() <= 3 / want * (2.0 ** -8 + 2.0 ** -18)
    assert int(torch.count_nonzero(t)) == 9


def test_version_of_written_tensors_moves():
    t = torch.ones(10, device=DEV)
    v = t._version
    B.sparge_clip_grads([t], 1.0)
    assert t._version > v


def test_refusals_on_the_device():
    a, b = torch.ones(64, device=DEV), torch.ones(64, device=DEV)
    for bad in (([],), ([a, a.cpu()],), ([a.half()],), ([a[::2]],), ([a.expand(2, 64)],)):
        with pytest.raises(ValueError):
            B.sparge_clip_grads(*bad, 1.0)
    for m in (float("inf"), float("nan"), -1.0):
        with pytest.raises(ValueError):
            B.sparge_clip_grads([a], m)
    with pytest.raises(ValueError):
        B.sparge_clip_grads([a, b], 1.0, out=[a])
    with pytest.raises(ValueError):
        B.sparge_clip_grads([a], 1.0, out=[a.bfloat16()])
    big = torch.ones(200, device=DEV)
    for ts, out in (([a, a], None), ([big[:64], big[60:124]], None), ([a, b], [big[:64], big[63:127]]),
                    ([a, b], [b, a]), ([big[:64], b], [big[32:96], b])):
        with pytest.raises(B.SpargeError) as e:
            B.sparge_clip_grads(ts, 1.0, out=out)
        assert e.value.code == B.SPARGE_ERR_INVALID_ARG
    assert (a == 1).all() and (b == 1).all() and (big == 1).all()
    # reading alone may overlap; an output may be its own input
    assert float(B.sparge_clip_grads([a, a], None)) == pytest.approx(math.sqrt(128), rel=1e-6)
    B.sparge_clip_grads([a, b], 1.0, out=[a, big[:64]])
    assert a[0] < 1 and b[0] == 1 and big[0] < 1 and big[64] == 1
    with pytest.raises(B.SpargeError) as e:
        B.sparge_clip_grads([a], 1.0, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    assert e.value.code == B.SPARGE_ERR_WORKSPACE
