"""Argument checks of the operators around the attention that need no GPU:
every call below fails validation before it reaches the device."""

import ctypes

import pytest
import torch

from block_sparse_attention_sparge_gb300 import binding as B

FAKE, ODD = 0x10000, 0x10008  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    return B.load_library(build_if_missing=True)


def _heads(**kw):
    a = B.Heads()
    a.B, a.N, a.d, a.n_parts, a.eps = 2, 100, 64, 1, 1e-6
    p = a.part[0]
    p.x, p.y, p.dx, p.H = FAKE, FAKE, FAKE, 4
    p.x_stride = p.dx_stride = (25600, 256, 64)
    for k, v in kw.items():
        setattr(p if hasattr(p, k) and not hasattr(a, k) else a, k, v)
    return a


def _rope(d=64):
    return B.RopeAxes(d, (d // 2, 0, 0))


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), B.SPARGE_ERR_INVALID_ARG), (dict(N=0), B.SPARGE_ERR_INVALID_ARG),
    (dict(n_parts=0), B.SPARGE_ERR_INVALID_ARG), (dict(n_parts=4), B.SPARGE_ERR_INVALID_ARG),
    (dict(n_parts=2), B.SPARGE_ERR_INVALID_ARG),  # an empty second part
    (dict(B=40000, N=30000), B.SPARGE_ERR_UNSUPPORTED), (dict(d=80), B.SPARGE_ERR_UNSUPPORTED),
    (dict(x_type=2), B.SPARGE_ERR_UNSUPPORTED), (dict(weight_type=-1), B.SPARGE_ERR_UNSUPPORTED),
    (dict(norm=3), B.SPARGE_ERR_INVALID_ARG), (dict(norm=-1), B.SPARGE_ERR_INVALID_ARG),
    (dict(eps=float("nan")), B.SPARGE_ERR_INVALID_ARG), (dict(eps=-1.0), B.SPARGE_ERR_INVALID_ARG),
    (dict(H=0), B.SPARGE_ERR_INVALID_ARG), (dict(H=129), B.SPARGE_ERR_UNSUPPORTED),
    (dict(y=None), B.SPARGE_ERR_INVALID_ARG), (dict(y=ODD), B.SPARGE_ERR_MISALIGNED),
    (dict(x=ODD, norm=1), B.SPARGE_ERR_MISALIGNED), (dict(x=None, norm=2), B.SPARGE_ERR_INVALID_ARG),
    (dict(x_stride=(25600, 260, 64), norm=1), B.SPARGE_ERR_MISALIGNED),
    (dict(x_stride=(25600, -256, 64), norm=1), B.SPARGE_ERR_INVALID_ARG),
    (dict(weight=ODD, norm=1), B.SPARGE_ERR_MISALIGNED),
    (dict(grid=FAKE), B.SPARGE_ERR_INVALID_ARG), (dict(pos=FAKE), B.SPARGE_ERR_INVALID_ARG),
])
def test_heads_checks(lib, kw, code):
    a = _heads(**kw)
    n = ctypes.c_size_t(0)
    assert lib.sparge_heads_fwd(ctypes.byref(a), None) == code
    assert lib.sparge_heads_bwd(ctypes.byref(a), None, 0, None) == code
    assert lib.sparge_heads_bwd_workspace_bytes(ctypes.byref(a), ctypes.byref(n)) == code


def test_heads_checks_of_rope_backward_and_workspace(lib):
    rope = _rope()
    at = ctypes.addressof(rope.plan)
    for kw in (dict(rope=at), dict(rope=at, grid=FAKE, pos=FAKE, pos_batch=1),
               dict(rope=at, pos=FAKE, pos_batch=3),
               dict(rope=ctypes.addressof(_keep(_rope(128)).plan), grid=FAKE)):
        a = _heads(**kw)
        assert lib.sparge_heads_fwd(ctypes.byref(a), None) == B.SPARGE_ERR_INVALID_ARG
    a = _heads(rope=at, grid=0x10002)
    assert lib.sparge_heads_fwd(ctypes.byref(a), None) == B.SPARGE_ERR_MISALIGNED
    bad = _rope()
    bad.plan.axis[5] = 3
    a = _heads(rope=ctypes.addressof(bad.plan), grid=FAKE)
    assert lib.sparge_heads_fwd(ctypes.byref(a), None) == B.SPARGE_ERR_INVALID_ARG
    assert lib.sparge_heads_fwd(None, None) == B.SPARGE_ERR_INVALID_ARG
    for kw, code in ((dict(dx=None), B.SPARGE_ERR_INVALID_ARG),
                     (dict(dx=ODD), B.SPARGE_ERR_MISALIGNED),
                     (dict(dx_stride=(25600, 256, 60)), B.SPARGE_ERR_MISALIGNED),
                     (dict(norm=1, dweight=0x10001), B.SPARGE_ERR_MISALIGNED),
                     (dict(norm=1, dweight=FAKE), B.SPARGE_ERR_WORKSPACE)):
        a = _heads(**kw)
        assert lib.sparge_heads_bwd(ctypes.byref(a), None, 0, None) == code, kw
    n = ctypes.c_size_t(0)
    a = _heads(norm=1, dweight=FAKE)
    assert lib.sparge_heads_bwd_workspace_bytes(ctypes.byref(a), ctypes.byref(n)) == 0
    assert n.value > 0 and n.value % (4 * 256) == 0  # rows of H * d sums
    assert lib.sparge_heads_bwd(ctypes.byref(a), FAKE, n.value - 1, None) == B.SPARGE_ERR_WORKSPACE
    assert lib.sparge_heads_bwd(ctypes.byref(a), ODD, n.value, None) == B.SPARGE_ERR_MISALIGNED
    for kw in (dict(), dict(norm=1), dict(norm=1, dweight=FAKE, plain=1)):
        a = _heads(**kw)
        assert lib.sparge_heads_bwd_workspace_bytes(ctypes.byref(a), ctypes.byref(n)) == 0
        assert n.value == 0
    assert lib.sparge_heads_bwd_workspace_bytes(ctypes.byref(a), None) == B.SPARGE_ERR_INVALID_ARG


_kept = []


def _keep(x):
    _kept.append(x)
    return x


def test_rope_plan(lib):
    r = B.RopeAxes(64, (12, 10, 10), theta=100.0, scale=(1.0, 0.5, -1.0), interleaved=False)
    assert list(r.plan.axis[:32]) == [0] * 12 + [1] * 10 + [2] * 10
    assert (r.plan.d, r.plan.interleaved) == (64, 0)
    two_pi = 6.283185307179586
    for j, (i, n, s) in enumerate([(i, 12, 1.0) for i in range(12)] + [(i, 10, 0.5) for i in range(10)]
                                  + [(i, 10, -1.0) for i in range(10)]):
        turns = s * 100.0 ** (-i / n) / two_pi
        frac = turns - (turns // 1)
        assert abs(r.plan.turn[j] / 2.0 ** 64 - frac) <= 2.0 ** -51  # four 64-bit roundings
    assert list(B.RopeAxes(64, (4,)).plan.turn[4:]) == [0] * 60
    assert B.RopeAxes(64, (1,), scale=(two_pi,)).plan.turn[0] in (0, 2 ** 64 - 2 ** 11, 2 ** 12)
    for bad in (dict(d=96, pairs=(1,)), dict(d=64, pairs=(20, 20)), dict(d=64, pairs=(-1,)),
                dict(d=64, pairs=(4,), theta=0.0), dict(d=64, pairs=(4,), theta=float("nan")),
                dict(d=64, pairs=(4,), scale=(float("inf"),))):
        with pytest.raises(B.SpargeError):
            B.RopeAxes(**bad)
    for bad in (dict(d=64, pairs=()), dict(d=64, pairs=(1, 1, 1, 1)),
                dict(d=64, pairs=(1, 1), scale=(1.0,))):
        with pytest.raises(ValueError):
            B.RopeAxes(**bad)
    assert lib.sparge_rope_init(None, 64, None, 1.0, None, 1) == B.SPARGE_ERR_INVALID_ARG


def test_rope_plan_survives_a_copy_of_its_owner(lib):
    """A copied plan points to its own memory, not to the original's."""
    import copy
    import pickle
    r = B.RopeAxes(64, (12, 10, 10), theta=77.0)
    for c in (copy.deepcopy(r), copy.copy(r), pickle.loads(pickle.dumps(r))):
        assert c.address == ctypes.addressof(c.plan)
        assert bytes(c.plan) == bytes(r.plan)
    assert copy.deepcopy(r).address != r.address


def _resnorm(**kw):
    a = B.Resnorm()
    a.rows, a.C, a.x_type, a.branch_type, a.norm, a.eps = 96, 256, 1, 0, 1, 1e-6
    a.gate_groups = a.scale_groups = a.shift_groups = 1
    for k in ("x", "branch", "y", "h", "stats", "dy", "dh", "dx", "dbranch"):
        setattr(a, k, FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


INV, UNS, MIS = B.SPARGE_ERR_INVALID_ARG, B.SPARGE_ERR_UNSUPPORTED, B.SPARGE_ERR_MISALIGNED


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), INV), (dict(C=0), INV), (dict(C=4), UNS), (dict(C=8200), UNS),
    (dict(rows=1 << 31), UNS), (dict(x_type=0, branch_type=1), UNS), (dict(x_type=2), UNS),
    (dict(norm=3), INV), (dict(eps=float("inf")), INV), (dict(norm=0, branch=None), INV),
    (dict(norm=0, scale=FAKE), INV), (dict(norm=0, shift=FAKE), INV),
    (dict(branch=None, gate=FAKE), INV), (dict(branch=None, post_weight=FAKE), INV),
    (dict(gate=ODD), MIS), (dict(gate=FAKE, gate_groups=0), INV),
    (dict(gate=FAKE, gate_groups=7), INV), (dict(gate=FAKE, gate_groups=4, gate_stride=-4), INV),
    (dict(gate=FAKE, gate_groups=4, gate_stride=258), MIS),
    (dict(gate=FAKE, gate_groups=4, gate_stride=256, shift=FAKE, shift_groups=2,
          shift_stride=256), UNS),
    (dict(x=ODD), MIS), (dict(x=None), INV), (dict(branch=ODD), MIS), (dict(post_weight=ODD), MIS),
])
def test_resnorm_checks(lib, kw, code):
    a = _resnorm(**kw)
    n = ctypes.c_size_t(0)
    assert lib.sparge_resnorm_fwd(ctypes.byref(a), None) == code
    assert lib.sparge_resnorm_bwd(ctypes.byref(a), None, 0, None) == code
    assert lib.sparge_resnorm_bwd_workspace_bytes(ctypes.byref(a), ctypes.byref(n)) == code


def test_resnorm_checks_of_each_direction(lib):
    for kw, code in ((dict(y=None), INV), (dict(y=ODD), MIS), (dict(h=None), INV),
                     (dict(stats=0x10002), MIS)):
        assert lib.sparge_resnorm_fwd(ctypes.byref(_resnorm(**kw)), None) == code, kw
    for kw, code in ((dict(stats=None), INV), (dict(dy=None, dh=None), INV), (dict(norm=0), INV),
                     (dict(dy=ODD), MIS), (dict(dh=ODD), MIS), (dict(dx=None), INV),
                     (dict(dbranch=None), INV), (dict(dgate=FAKE), INV), (dict(dpost=FAKE), INV),
                     (dict(gate=FAKE, dgate=ODD), MIS),
                     (dict(gate=FAKE, dgate=FAKE), B.SPARGE_ERR_WORKSPACE)):
        a = _resnorm(**kw)
        assert lib.sparge_resnorm_bwd(ctypes.byref(a), None, 0, None) == code, kw
    a = _resnorm(gate=FAKE, dgate=FAKE)
    n = ctypes.c_size_t(0)
    assert lib.sparge_resnorm_bwd_workspace_bytes(ctypes.byref(a), ctypes.byref(n)) == 0
    assert lib.sparge_resnorm_bwd(ctypes.byref(a), FAKE, n.value - 1, None) == B.SPARGE_ERR_WORKSPACE
    assert lib.sparge_resnorm_bwd(ctypes.byref(a), ODD, n.value, None) == MIS
    assert lib.sparge_resnorm_bwd_workspace_bytes(ctypes.byref(_resnorm()), ctypes.byref(n)) == 0
    assert n.value == 0  # no sums wanted
    assert lib.sparge_resnorm_fwd(None, None) == INV


def test_clip_checks(lib):
    def call(rows, out=None, max_norm=1.0, eps=1e-6, norm=FAKE, ws=FAKE, size=1 << 20, n=None):
        import array
        table = array.array("q", [v for r in rows for v in r])
        outs = array.array("q", out) if out is not None else None
        return lib.sparge_clip_grads(table.buffer_info()[0], outs.buffer_info()[0] if outs else None,
                                     len(rows) if n is None else n, max_norm, eps, norm, ws, size,
                                     None)
    one = [(FAKE, 100, 0)]
    assert call(one, n=-1) == INV
    assert call(one, n=65537) == UNS
    for kw in (dict(max_norm=float("nan")), dict(max_norm=float("inf")), dict(eps=-1.0),
               dict(eps=float("nan")), dict(norm=None)):
        assert call(one, **kw) == INV
    assert call(one, norm=0x10001) == MIS
    assert call([(FAKE, 100, 2)]) == UNS
    assert call([(FAKE, -1, 0)]) == INV
    assert call([(FAKE, 1 << 41, 0)]) == UNS
    assert call([(0, 5, 0)]) == INV
    assert call(one, out=[0]) == INV
    assert call([(FAKE + 1, 5, 0)]) == MIS
    assert call([(FAKE + 2, 5, 1)]) == MIS
    assert call(one, out=[FAKE + 1001]) == MIS
    # overlaps: twice, by one value, an output on another input, on its own shifted
    assert call(one * 2) == INV
    assert call([(FAKE, 100, 0), (FAKE + 198, 5, 0)]) == INV
    assert call([(FAKE, 100, 0), (FAKE + 200, 5, 0)], ws=None) == B.SPARGE_ERR_WORKSPACE
    assert call([(FAKE, 100, 0), (FAKE + 4096, 100, 0)], out=[FAKE + 4096, FAKE + 8192]) == INV
    assert call(one, out=[FAKE + 2]) == INV
    assert call([(FAKE, 100, 0), (FAKE + 4096, 100, 1)], out=[FAKE + 9000, FAKE + 9196]) == INV
    assert call(one, out=[FAKE], ws=None) == B.SPARGE_ERR_WORKSPACE
    assert call(one * 2, max_norm=-1.0, ws=None) == B.SPARGE_ERR_WORKSPACE  # reading may overlap
    assert call(one, size=1) == B.SPARGE_ERR_WORKSPACE
    assert call(one, ws=ODD) == MIS
    n = ctypes.c_size_t(0)
    assert lib.sparge_clip_workspace_bytes(1, ctypes.byref(n)) == 0 and n.value > 0
    one_list = n.value
    assert lib.sparge_clip_workspace_bytes(1024, ctypes.byref(n)) == 0 and n.value == one_list
    assert lib.sparge_clip_workspace_bytes(1025, ctypes.byref(n)) == 0 and n.value == 2 * one_list
    assert lib.sparge_clip_workspace_bytes(-1, ctypes.byref(n)) == INV


def test_structs_match_the_header():
    """Sizes of the C structs on every 64-bit platform this builds on."""
    assert ctypes.sizeof(B.Rope) == 584
    assert ctypes.sizeof(B.HeadsPart) == 96
    assert ctypes.sizeof(B.Heads) == 352
    assert ctypes.sizeof(B.Resnorm) == 208
    assert (B._HEADS.size, B._RESNORM.size) == (352, 208)


def test_cpu_tensors_are_refused():
    q = torch.zeros(1, 8, 2, 64)
    x = torch.zeros(1, 8, 64)
    for call in (lambda: B.sparge_heads_fwd(q), lambda: B.sparge_heads_fwd(),
                 lambda: B.sparge_heads_bwd(q.bfloat16()), lambda: B.sparge_heads_bwd(),
                 lambda: B.sparge_resnorm_fwd(x), lambda: B.sparge_resnorm_bwd(x, None, x),
                 lambda: B.sparge_clip_grads([x], 1.0), lambda: B.sparge_clip_grads([], 1.0)):
        with pytest.raises(ValueError):
            call()
