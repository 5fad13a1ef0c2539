"""Head layout with RMS norm and rotary positions (sparge_heads_fwd / _bwd)
against the 64-bit form."""

import pytest
import torch

import block_reference as R
from block_sparse_attention_sparge_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _pairs(d):
    return (d // 2 - 2 * (d // 6), d // 6, d // 6)


def _rand(g, *shape, dtype=BF, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g) * std + mean).to(dtype)


def _make(b, n, h, d, dtype, norm, seed=0, w_dtype=None):
    g = _gen(seed)
    q, k, v = (_rand(g, b, n, h, d, dtype=dtype, std=1.5) for _ in range(3))
    width = {None: 0, "token": h * d, "head": d}[norm]
    wq, wk = ((_rand(g, width, dtype=w_dtype or dtype, std=0.2, mean=1.0) if width else None)
              for _ in range(2))
    return q, k, v, wq, wk


def _dev(*ts):
    return tuple(None if t is None else t.to(DEV) for t in ts)


def _check_fwd(got, x, w, norm, cs, inter, eps=1e-6, what=""):
    ref, bound = R.heads_fwd(R.f64(x), R.f64(w), norm, cs, inter, eps)
    R.check(got, ref, bound, what)


CASES = [
    # b, n, heads, d, type, norm, interleaved, grid of the first sample
    (1, 1, 1, 64, BF, "token", True, (1, 1, 1)),
    (1, 1, 1, 128, F32, "head", False, (1, 1, 1)),
    (2, 33, 3, 64, BF, "head", True, (2, 3, 5)),      # padding behind the grid
    (1, 60, 2, 128, BF, None, False, (3, 4, 5)),
    (3, 7, 5, 64, F32, "token", False, (7, 1, 1)),
    (1, 131, 12, 128, BF, "token", True, (5, 5, 5)),
    (1, 50, 7, 64, F32, "token", True, (2, 5, 5)),
    (1, 29, 40, 128, BF, "token", False, (1, 4, 7)),  # 640 threads a row
    (1, 11, 64, 128, F32, "head", True, (1, 2, 5)),   # 1024 threads a row
    (1, 9, 63, 128, BF, "token", False, (3, 3, 1)),
    (1, 6000, 1, 64, BF, "head", False, (15, 20, 20)),  # many rows a slot
    (2, 3001, 9, 128, BF, "token", True, (6, 25, 20)),
    # a norm over each head of full rows
    (2, 301, 4, 128, BF, "head", True, (6, 7, 7)),
    (1, 2, 2, 128, F32, "head", False, (1, 1, 2)),
    (3, 1501, 12, 128, BF, "head", False, (15, 10, 10)),
    (1, 77, 12, 128, F32, "head", True, (7, 11, 1)),
    (2, 301, 40, 128, BF, "head", True, (6, 7, 7)),
    (1, 333, 40, 128, BF, "head", False, (3, 10, 11)),
    (1, 45, 40, 128, F32, "head", False, (3, 3, 5)),
    (1, 9, 64, 128, BF, "head", True, (3, 3, 1)),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c[:4]))
def test_forward_and_backward(case):
    b, n, h, d, dtype, norm, inter, grid0 = case
    q, k, v, wq, wk = _make(b, n, h, d, dtype, norm)
    grid = torch.tensor([[max(1, grid0[0] - i), grid0[1], grid0[2]] for i in range(b)],
                        dtype=torch.int32)
    rope = B.RopeAxes(d, _pairs(d), interleaved=inter)
    cs = R.angles(R.positions(b, n, grid), _pairs(d), d)
    how = dict(rope=rope, grid=grid.to(DEV), norm=norm, q_weight=None, k_weight=None)
    how["q_weight"], how["k_weight"] = _dev(wq, wk)
    got = B.sparge_heads_fwd(*_dev(q, k, v), **how)
    for name, y, x, w in (("q", got[0], q, wq), ("k", got[1], k, wk)):
        _check_fwd(y, x, w, norm, cs, inter, what=name)
    assert torch.equal(got[2].cpu(), v.to(BF).transpose(1, 2))

    g = _gen(9)
    dq, dk, dv = (_rand(g, b, h, n, d) for _ in range(3))
    grads = B.sparge_heads_bwd(*_dev(dq, dk, dv, q, k), **how)
    for name, i, dy, x, w in (("q", 0, dq, q, wq), ("k", 1, dk, k, wk)):
        dx, bound, dw, dwb = R.heads_bwd(R.f64(dy), R.f64(x), R.f64(w), norm, cs, inter)
        R.check(grads[i], dx, bound, "d" + name)
        assert grads[i].dtype == dtype
        if norm is None:
            assert grads[3 + i] is None
        else:
            R.check(grads[3 + i], dw, dwb, "dw" + name)
    assert torch.equal(grads[2].cpu(), dv.to(dtype).transpose(1, 2))
    again = B.sparge_heads_bwd(*_dev(dq, dk, dv, q, k), **how)
    for x, y in zip(grads, again):
        assert x is None or torch.equal(x, y)


@pytest.mark.parametrize("given", [False, True], ids=["grid", "pos"])
@pytest.mark.parametrize("case", [(6000, 1, 2, 64, BF, "head"), (700, 5, 12, 128, BF, "token"),
                                  (900, 4, 3, 64, F32, "token"), (350, 3, 20, 128, F32, "token")],
                         ids=lambda c: "-".join(str(x) for x in c[:4]))
def test_steps_over_several_samples(case, given):
    """More short samples than the machine has slots: a slot's next token lies
    samples further on."""
    b, n, h, d, dtype, norm = case
    q, k, v, wq, wk = _make(b, n, h, d, dtype, norm, seed=3)
    g = _gen(6)
    rope = B.RopeAxes(d, _pairs(d))
    how = dict(rope=rope, norm=norm)
    how["q_weight"], how["k_weight"] = _dev(wq, wk)
    if given:
        pos = torch.randint(-9, 2000, (b, n, 3), generator=g, dtype=torch.int32)
        how["pos"] = pos.to(DEV)
        at = pos.double()
    else:
        grid = torch.randint(1, 4, (b, 3), generator=g, dtype=torch.int32)
        how["grid"] = grid.to(DEV)
        at = R.positions(b, n, grid)
    cs = R.angles(at, _pairs(d), d)
    got = B.sparge_heads_fwd(*_dev(q, k, v), **how)
    _check_fwd(got[0], q, wq, norm, cs, True)
    _check_fwd(got[1], k, wk, norm, cs, True)
    assert torch.equal(got[2].cpu(), v.to(BF).transpose(1, 2))
    dq, dk, dv = (_rand(g, b, h, n, d) for _ in range(3))
    grads = B.sparge_heads_bwd(*_dev(dq, dk, dv, q, k), **how)
    for i, dy, x, w in ((0, dq, q, wq), (1, dk, k, wk)):
        dx, bound, dw, dwb = R.heads_bwd(R.f64(dy), R.f64(x), R.f64(w), norm, cs, True)
        R.check(grads[i], dx, bound)
        R.check(grads[3 + i], dw, dwb)
    assert torch.equal(grads[2].cpu(), dv.to(dtype).transpose(1, 2))


@pytest.mark.parametrize("norm", ["token", "head"])
def test_steps_over_several_samples_with_few_key_heads(norm):
    b, n, d = 900, 5, 64
    g = _gen(8)
    q, k, v = (_rand(g, b, n, h, d) for h in (12, 3, 5))
    grid = torch.randint(1, 4, (b, 3), generator=g, dtype=torch.int32)
    rope = B.RopeAxes(d, _pairs(d), interleaved=False)
    cs = R.angles(R.positions(b, n, grid), _pairs(d), d)
    how = dict(rope=rope, grid=grid.to(DEV), norm=norm)
    got = B.sparge_heads_fwd(*_dev(q, k, v), **how)
    _check_fwd(got[0], q, None, norm, cs, False)
    _check_fwd(got[1], k, None, norm, cs, False)
    assert torch.equal(got[2].cpu(), v.transpose(1, 2))
    dq, dk, dv = (_rand(g, b, h, n, d) for h in (12, 3, 5))
    grads = B.sparge_heads_bwd(*_dev(dq, dk, dv, q, k), **how)
    for i, dy, x in ((0, dq, q), (1, dk, k)):
        dx, bound, _, _ = R.heads_bwd(R.f64(dy), R.f64(x), None, norm, cs, False)
        R.check(grads[i], dx, bound)
    assert torch.equal(grads[2].cpu(), dv.transpose(1, 2))


@pytest.mark.parametrize("norm", ["token", "head"])
def test_norm_weight_type_apart_from_the_input_type_and_no_weight(norm):
    q, k, v, wq, _ = _make(1, 19, 3, 64, BF, norm, w_dtype=F32)
    qd, kd, wd = _dev(q, k, wq)
    got = B.sparge_heads_fwd(qd, kd, norm=norm, q_weight=wd)
    assert got[2] is None
    _check_fwd(got[0], q, wq, norm, None, True)
    _check_fwd(got[1], k, None, norm, None, True)
    dq = _rand(_gen(1), 1, 3, 19, 64)
    res = B.sparge_heads_bwd(dq.to(DEV), None, None, qd, norm=norm, q_weight=wd)
    dx, bound, dw, dwb = R.heads_bwd(R.f64(dq), R.f64(q), R.f64(wq), norm, None, True)
    R.check(res[0], dx, bound)
    R.check(res[3], dw, dwb)
    assert res[3].dtype == F32 and res[1] is res[2] is res[4] is None


@pytest.mark.parametrize("dtype", [BF, F32])
def test_slices_of_a_fused_projection_and_other_orders(dtype):
    b, n, h, d = 2, 37, 3, 64
    g = _gen(4)
    qkv = _rand(g, b, n, 3 * h * d + 16, dtype=dtype)
    dev = qkv.to(DEV)
    parts = [dev[..., 8 + i * h * d:8 + (i + 1) * h * d].unflatten(-1, (h, d)) for i in range(3)]
    host = [qkv[..., 8 + i * h * d:8 + (i + 1) * h * d].unflatten(-1, (h, d)) for i in range(3)]
    got = B.sparge_heads_fwd(*parts, norm="token")
    for i in range(2):
        _check_fwd(got[i], host[i], None, "token", None, True)
    assert torch.equal(got[2].cpu(), host[2].to(BF).transpose(1, 2))
    # heads outermost in memory, tokens before samples
    x = _rand(g, h, n, b, d, dtype=dtype)
    y = B.sparge_heads_fwd(x.to(DEV).permute(2, 1, 0, 3), norm="head")[0]
    _check_fwd(y, x.permute(2, 1, 0, 3), None, "head", None, True)
    # a sample shared by the batch
    x1 = x.permute(2, 1, 0, 3)[:1]
    y = B.sparge_heads_fwd(x1.to(DEV).expand(b, n, h, d))[0]
    assert torch.equal(y.cpu(), x1.expand(b, n, h, d).to(BF).transpose(1, 2))
    # gradients into slices: nothing else of the buffer is touched
    buf = torch.full((b, n, 3 * h * d + 16), 7.0, dtype=dtype, device=DEV)
    out = [buf[..., 8 + i * h * d:8 + (i + 1) * h * d].unflatten(-1, (h, d)) for i in range(3)]
    dys = [_rand(g, b, h, n, d) for _ in range(3)]
    B.sparge_heads_bwd(*_dev(*dys), parts[0], parts[1], norm="token", out=out)
    for i in range(2):
        dx, bound, _, _ = R.heads_bwd(R.f64(dys[i]), R.f64(host[i]), None, "token", None, True)
        R.check(out[i], dx, bound)
    assert torch.equal(out[2].cpu(), dys[2].to(dtype).transpose(1, 2))
    assert (buf[..., :8] == 7).all() and (buf[..., 8 + 3 * h * d:] == 7).all()


def test_heads_of_different_number_share_a_launch():
    """One wide part (1024 threads a row) beside a narrow one (8 slots)."""
    g = _gen(5)
    q, k, v = _rand(g, 1, 21, 64, 128), _rand(g, 1, 21, 1, 128), _rand(g, 1, 21, 2, 128)
    grid = torch.tensor([[1, 4, 5]], dtype=torch.int32)
    cs = R.angles(R.positions(1, 21, grid), _pairs(128), 128)
    rope = B.RopeAxes(128, _pairs(128))
    for norm in ("token", "head"):
        got = B.sparge_heads_fwd(*_dev(q, k, v), rope=rope, grid=grid.to(DEV), norm=norm)
        _check_fwd(got[0], q, None, norm, cs, True)
        _check_fwd(got[1], k, None, norm, cs, True)
        assert torch.equal(got[2].cpu(), v.transpose(1, 2))
        dq, dk, dv = (_rand(g, 1, t.shape[2], 21, 128) for t in (q, k, v))
        w = torch.ones(128 if norm == "head" else 64 * 128, dtype=BF)
        wk = torch.ones(128, dtype=BF)
        res = B.sparge_heads_bwd(*_dev(dq, dk, dv, q, k), rope=rope, grid=grid.to(DEV), norm=norm,
                                 q_weight=w.to(DEV), k_weight=wk.to(DEV))
        for i, (dy, x, ww) in enumerate(((dq, q, w), (dk, k, wk))):
            dx, bound, dw, dwb = R.heads_bwd(R.f64(dy), R.f64(x), R.f64(ww), norm, cs, True)
            R.check(res[i], dx, bound)
            R.check(res[3 + i], dw, dwb)


@pytest.mark.parametrize("shared", [True, False])
@pytest.mark.parametrize("interleaved", [True, False])
def test_positions_given_per_token(shared, interleaved):
    b, n, h, d = 2, 41, 2, 64
    q, k, _, _, _ = _make(b, n, h, d, F32, None, seed=6)
    pairs, scale, theta = (5, 20, 3), (0.5, 1.0, 2.25), 500.0  # 4 pairs do not turn
    pos = torch.randint(-1000000, 1000000, (1 if shared else b, n, 3), generator=_gen(7))
    pos[0, 0] = 0
    rope = B.RopeAxes(d, pairs, theta, scale, interleaved)
    cs = R.angles(R.positions(b, n, pos=pos), pairs, d, theta, scale)
    got = B.sparge_heads_fwd(*_dev(q, k), rope=rope, pos=pos.to(DEV, torch.int32))
    _check_fwd(got[0], q, None, None, cs, interleaved)
    _check_fwd(got[1], k, None, None, cs, interleaved)
    assert torch.equal(got[0][0, :, 0].cpu(), q[0, 0].to(BF))  # position 0 turns nothing


def test_rotation_by_the_largest_positions():
    """At +-2^31 the product of position and frequency is reduced exactly; what
    is left is the 64-bit error of the frequencies times the position."""
    d, n = 64, 6
    lim = 2 ** 31
    pos = torch.tensor([lim - 1, -lim, lim - 2, 1 - lim, 2 ** 30 + 1, -(2 ** 24) - 1])
    pos = pos[:, None].expand(n, 3)[None].contiguous()
    q = _rand(_gen(8), 1, n, 1, d, dtype=F32)
    got = B.sparge_heads_fwd(q.to(DEV), rope=B.RopeAxes(d, _pairs(d)),
                             pos=pos.to(DEV, torch.int32))[0]
    cs = R.angles(R.positions(1, n, pos=pos), _pairs(d), d)
    ref, bound = R.heads_fwd(R.f64(q), None, None, cs, True)
    # the kernel's frequency: power (2^-52) and two products (2^-53 each); the
    # reference's: power and one product; in all 7 * 2^-53 of the angle
    R.check(got, ref, bound + 8 * lim * 2.0 ** -53 * R.pair_size(R.f64(q), True).transpose(1, 2))


def test_grids_that_cover_nothing_or_more_than_the_tokens():
    b, n, d = 6, 23, 64
    q = _rand(_gen(10), b, n, 2, d, dtype=F32)
    big = 2 ** 31 - 1
    grid = torch.tensor([[0, 4, 4], [3, -1, 4], [-2, -2, 4], [big, big, big], [big, 1, 3],
                         [4, 2, 2]], dtype=torch.int32)
    rope = B.RopeAxes(d, _pairs(d))
    got = B.sparge_heads_fwd(q.to(DEV), rope=rope, grid=grid.to(DEV))[0]
    for s in range(3):
        assert torch.equal(got[s].cpu(), q[s].to(BF).transpose(0, 1))
    cs = R.angles(R.positions(b, n, grid), _pairs(d), d)
    _check_fwd(got, q, None, None, cs, True)
    assert torch.equal(got[5][:, 16:].cpu(), q[5, 16:].to(BF).transpose(0, 1))  # padding


def test_rows_of_infinities_nan_and_zeros_stay_alone():
    q = _rand(_gen(11), 1, 12, 3, 64, dtype=F32)
    q[0, 2] = 0.0
    q[0, 5, 1, 7] = float("inf")
    q[0, 8, 0, 0] = float("nan")
    got = B.sparge_heads_fwd(q.to(DEV), norm="token")[0].cpu()
    assert (got[:, :, 2] == 0).all()
    assert got[0, 1, 5, 7].isnan() and (got[0, 0, 5] == 0).all()
    assert got[0, :, 8].isnan().all()
    keep = [i for i in range(12) if i not in (5, 8)]
    ref, bound = R.heads_fwd(R.f64(q)[:, keep], None, "token", None, True)
    R.check(got[:, :, keep], ref, bound)


def test_against_differences():
    """<gradient, v> against central differences of the 64-bit forward.  The
    step 2^-10 leaves a third-order error below 2^-20 of the sizes used."""
    b, n, h, d = 1, 13, 2, 64
    for norm in ("token", "head"):
        q, _, _, w, _ = _make(b, n, h, d, F32, norm, seed=12)
        grid = torch.tensor([[1, 3, 4]], dtype=torch.int32)
        cs = R.angles(R.positions(b, n, grid), _pairs(d), d)
        dq = _rand(_gen(13), b, h, n, d)
        res = B.sparge_heads_bwd(dq.to(DEV), None, None, q.to(DEV), rope=B.RopeAxes(d, _pairs(d)),
                                 grid=grid.to(DEV), norm=norm, q_weight=w.to(DEV))
        vx, vw = (torch.randn(t.shape, generator=_gen(14), dtype=torch.float64) for t in (q, w))

        def loss(e, which):
            x, ww = R.f64(q), R.f64(w)
            x, ww = (x + e * vx, ww) if which == 0 else (x, ww + e * vw)
            return float((R.heads_fwd(x, ww, norm, cs, True)[0] * R.f64(dq)).sum())

        _, bx, _, bw = R.heads_bwd(R.f64(dq), R.f64(q), R.f64(w), norm, cs, True)
        e = 2.0 ** -10
        for which, got, v, bound in ((0, res[0], vx, bx), (1, res[3], vw, bw)):
            diff = (loss(e, which) - loss(-e, which)) / (2 * e)
            dot = float((R.f64(got) * v).sum())
            room = float((bound * v.abs()).sum()) + 2.0 ** -18 * float((R.f64(got) * v).abs().sum())
            assert abs(dot - diff) <= room, (norm, which, dot, diff, room)


def test_out_and_its_surroundings_and_stream_order():
    b, n, h, d = 1, 77, 3, 64
    q, k, v, w, _ = _make(b, n, h, d, BF, "token", seed=15)
    qd, kd, vd, wd = _dev(q, k, v, w)
    ref = B.sparge_heads_fwd(qd, kd, vd, norm="token", q_weight=wd)
    size = b * h * n * d
    buf = torch.full((3 * size + 64,), 5.0, dtype=BF, device=DEV)
    out = [buf[16 + i * (size + 16):][:size].view(b, h, n, d) for i in range(3)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        late = qd.clone().zero_()
        torch.cuda._sleep(20_000_000)
        late.copy_(qd)
        got = B.sparge_heads_fwd(late, kd, vd, norm="token", q_weight=wd, out=out)
    stream.synchronize()
    for r, o, g in zip(ref, out, got):
        assert g is o and torch.equal(r, o)
    for i in range(4):
        assert (buf[i * (size + 16):][:16] == 5).all()


def test_captured_and_replayed():
    b, n, h, d = 1, 500, 4, 128
    q, k, v, wq, wk = _make(b, n, h, d, BF, "token", seed=16)
    qd, kd, vd, wqd, wkd = _dev(q, k, v, wq, wk)
    dys = _dev(*(_rand(_gen(17 + i), b, h, n, d) for i in range(3)))
    grid = torch.tensor([[5, 10, 10]], dtype=torch.int32, device=DEV)
    how = dict(rope=B.RopeAxes(d, _pairs(d)), grid=grid, norm="token", q_weight=wqd, k_weight=wkd)
    B.sparge_heads_fwd(qd, kd, vd, **how)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fwd = B.sparge_heads_fwd(qd, kd, vd, **how)
        bwd = B.sparge_heads_bwd(*dys, qd, kd, **how)
    for seed in (20, 21):
        new = _make(b, n, h, d, BF, "token", seed=seed)
        for t, s in zip((qd, kd, vd, wqd, wkd), new):
            t.copy_(s)
        grid.copy_(torch.tensor([[seed - 18, 9, 9]], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((*fwd, *bwd), (*B.sparge_heads_fwd(qd, kd, vd, **how),
                                       *B.sparge_heads_bwd(*dys, qd, kd, **how))):
            assert torch.equal(x, y)


def test_offsets_past_32_bits():
    """2.3e9 elements between the first and the last token."""
    n, h, d = 150001, 40, 128
    c = h * d
    qkv = torch.zeros((1, n, 3 * c), dtype=BF, device=DEV)
    assert qkv.numel() > 2 ** 31
    rows = [0, 1, 139811, n - 2, n - 1]  # 139811: behind element 2^31
    qkv[:, rows] = _rand(_gen(22), 1, len(rows), 3 * c).to(DEV)
    parts = [qkv[..., i * c:(i + 1) * c].unflatten(-1, (h, d)) for i in range(3)]
    pos = torch.arange(n, dtype=torch.int32, device=DEV)[None, :, None].expand(1, n, 3).contiguous()
    rope = B.RopeAxes(d, _pairs(d))
    got = B.sparge_heads_fwd(*parts, rope=rope, pos=pos, norm="token")
    cs = R.angles(R.positions(1, len(rows), pos=pos[:, rows]), _pairs(d), d)
    for i in range(2):
        _check_fwd(got[i][:, :, rows], parts[i][:, rows], None, "token", cs, True)
        assert int(torch.count_nonzero(got[i].amax((1, 3)))) == len(rows)
    assert torch.equal(got[2][:, :, rows], parts[2][:, rows].transpose(1, 2))
    out = torch.zeros_like(qkv)
    outs = [out[..., i * c:(i + 1) * c].unflatten(-1, (h, d)) for i in range(3)]
    B.sparge_heads_bwd(*got, rope=rope, pos=pos, out=outs)
    for i in range(2):
        dx, bound, _, _ = R.heads_bwd(R.f64(got[i][:, :, rows]), None, None, None, cs, True)
        R.check(outs[i][:, rows], dx, bound)
    assert torch.equal(outs[2][:, rows], parts[2][:, rows])


def test_refusals_on_the_device():
    q = torch.zeros(1, 8, 2, 64, dtype=BF, device=DEV)
    rope = B.RopeAxes(64, (12, 10, 10))
    grid = torch.ones(1, 3, dtype=torch.int32, device=DEV)
    with pytest.raises(B.SpargeError) as e:
        B.sparge_heads_fwd(torch.zeros(1, 8, 129, 64, dtype=BF, device=DEV))
    assert e.value.code == B.SPARGE_ERR_UNSUPPORTED
    with pytest.raises(B.SpargeError) as e:
        B.sparge_heads_fwd(torch.zeros(1, 8, 2, 96, dtype=BF, device=DEV))
    assert e.value.code == B.SPARGE_ERR_UNSUPPORTED
    with pytest.raises(B.SpargeError) as e:
        B.sparge_heads_fwd(torch.zeros(1, 0, 2, 64, dtype=BF, device=DEV))
    assert e.value.code == B.SPARGE_ERR_INVALID_ARG
    odd = torch.zeros(1, 8, 2 * 64 + 4, dtype=BF, device=DEV)
    for x in (odd[..., 4:].unflatten(-1, (2, 64)), odd[..., :128].unflatten(-1, (2, 64))):
        with pytest.raises(B.SpargeError) as e:
            B.sparge_heads_fwd(x)
        assert e.value.code == B.SPARGE_ERR_MISALIGNED
    for bad in (dict(rope=rope), dict(grid=grid), dict(rope=rope, grid=grid, pos=grid[None]),
                dict(rope=B.RopeAxes(128, (22, 21, 21)), grid=grid),
                dict(rope=rope, grid=grid.long()), dict(rope=rope, grid=grid.repeat(2, 1)),
                dict(norm="row"), dict(q_weight=torch.ones(64, device=DEV)),
                dict(norm="head", q_weight=torch.ones(128, device=DEV)),
                dict(norm="head", k_weight=torch.ones(64, device=DEV)),
                dict(norm="head", q_weight=torch.ones(64, device=DEV, dtype=torch.float16)),
                dict(rope=rope, pos=torch.zeros(1, 7, 3, dtype=torch.int32, device=DEV)),
                dict(k=torch.zeros(1, 9, 2, 64, dtype=BF, device=DEV)),
                dict(k=torch.zeros(1, 8, 2, 64, device=DEV)),
                dict(k=torch.zeros(1, 8, 2, 64, dtype=BF))):
        with pytest.raises(ValueError):
            B.sparge_heads_fwd(q, **bad)
    with pytest.raises(ValueError):
        B.sparge_heads_fwd(q.half())
    with pytest.raises(ValueError):
        B.sparge_heads_fwd(q[..., ::2])
    dq = torch.zeros(1, 2, 8, 64, dtype=BF, device=DEV)
    for bad in (dict(norm="token"), dict(out=(q.float(), None, None), q=q),
                dict(out=(torch.zeros(1, 8, 1, 64, dtype=BF, device=DEV).expand(1, 8, 2, 64),
                          None, None)),
                dict(norm="token", q=q[:, :4])):
        with pytest.raises(ValueError):
            B.sparge_heads_bwd(dq, **bad)
    same = torch.zeros(1, 8, 2, 64, dtype=BF, device=DEV)
    with pytest.raises(ValueError):
        B.sparge_heads_bwd(dq, dq, out=(same, same, None))
    with pytest.raises(ValueError):
        B.sparge_heads_fwd(q, q, out=(dq, dq, None))
    with pytest.raises(B.SpargeError) as e:
        B.sparge_heads_bwd(dq, q=q, norm="head", q_weight=torch.ones(64, device=DEV),
                           workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.code == B.SPARGE_ERR_WORKSPACE
