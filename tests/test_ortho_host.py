"""Argument checks of the orthogonalised updates that need no GPU: every call
below fails validation before it reaches the device."""

import ctypes

import pytest
import torch

from block_sparse_attention_sparge_gb300 import binding as B

FAKE = 1 << 20  # never dereferenced
INV, UNS, MIS = B.SPARGE_ERR_INVALID_ARG, B.SPARGE_ERR_UNSUPPORTED, B.SPARGE_ERR_MISALIGNED
WS = B.SPARGE_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    return B.load_library(build_if_missing=True)


def _args(rows=({},), **kw):
    table = (B.Matrix * max(1, len(rows)))()
    for i, m in enumerate(rows):
        t = table[i]
        t.rows, t.cols, t.grad_stride, t.out_stride, t.momentum_stride = 20, 30, 30, 30, 30
        t.grad_type = t.out_type = 1
        t.grad, t.out = (FAKE << 4) + 65536 * i, (FAKE << 8) + 65536 * i
        for k, v in m.items():
            setattr(t, k, v)
    a = B.Ortho()
    a.mats, a.n, a.steps = ctypes.addressof(table), len(rows), 5
    a.a, a.b, a.c, a.eps = 3.4445, -4.7750, 2.0315, 1e-7
    for k, v in kw.items():
        setattr(a, k, v)
    a._hold = table
    return a


def test_structs_match_the_header():
    assert ctypes.sizeof(B.Matrix) == 72 == B._MATRIX.size
    assert ctypes.sizeof(B.Ortho) == 56 == B._ORTHO.size


@pytest.mark.parametrize("rows,kw,code", [
    ((), {}, INV), (({},), dict(mats=0), INV), (({},), dict(n=-1), INV), (({},), dict(n=65537), UNS),
    ((dict(rows=0),), {}, INV), ((dict(cols=-3),), {}, INV), ((dict(rows=65537),), {}, UNS),
    (({}, dict(cols=70000)), {}, UNS),
    ((dict(grad=0),), {}, INV), ((dict(out=0),), {}, INV), ((dict(grad=FAKE + 2),), {}, MIS),
    ((dict(out=FAKE + 1, out_type=0),), {}, MIS), ((dict(momentum=FAKE + 2),), {}, MIS),
    ((dict(grad_type=2),), {}, UNS), ((dict(out_type=-1),), {}, UNS),
    ((dict(grad_stride=0),), {}, INV), ((dict(grad_stride=-30),), {}, INV),
    ((dict(out_stride=20),), {}, INV),  # rows that overlap
    ((dict(out_stride=1 << 50),), {}, INV),
    ((dict(keep=float("nan")),), {}, INV), ((dict(step=float("inf")),), {}, INV),
    (({},), dict(steps=-1), INV), (({},), dict(steps=65), INV), (({},), dict(a=17.0), INV),
    (({},), dict(b=float("nan")), INV), (({},), dict(c=float("-inf")), INV),
    (({},), dict(eps=-1.0), INV), (({},), dict(eps=float("inf")), INV),
    (({},), dict(mu=float("nan")), INV), (({},), dict(status=FAKE + 2), MIS),
    # shared memory
    ((dict(out=(FAKE << 4) + 4),), {}, INV), ((dict(out=FAKE << 4),), dict(update=1), INV),
    ((dict(momentum=FAKE << 4),), {}, INV), ((dict(momentum=FAKE << 8),), {}, INV),
    ((dict(out=FAKE << 9), dict(out=(FAKE << 9) + 2396)), {}, INV),
    (({}, dict(grad=FAKE << 8)), {}, INV), (({}, dict(momentum=(FAKE << 4) + 128)), {}, INV),
    # in its own place, beside one another, and the same gradient twice
    ((dict(out=FAKE << 4),), {}, WS), ((dict(out=FAKE << 9), dict(out=(FAKE << 9) + 2400)), {}, WS),
    ((dict(out=FAKE << 9, out_stride=60), dict(out=(FAKE << 9) + 120, out_stride=60)), {}, WS),
    ((dict(grad=FAKE << 5), dict(grad=FAKE << 5)), {}, WS),
    ((dict(rows=1, grad_stride=-5, out_stride=0),), {}, WS),
    (({},), {}, WS),
])
def test_checks(lib, rows, kw, code):
    assert lib.sparge_orthogonalize(ctypes.byref(_args(rows, **kw)), None, 0, None) == code


def test_workspace(lib):
    n = ctypes.c_size_t(0)
    f = lib.sparge_orthogonalize_workspace_bytes
    assert f(ctypes.byref(_args()), None) == INV
    assert f(None, ctypes.byref(n)) == INV
    assert lib.sparge_orthogonalize(None, None, 0, None) == INV
    assert f(ctypes.byref(_args(half=1)), ctypes.byref(n)) == 0
    # X twice in two planes, A and B, of 128 x 128 fp16 values, and fp32 vectors
    one = 6 * 32768 + 16384
    assert one < n.value <= one + 256 * 8
    assert f(ctypes.byref(_args()), ctypes.byref(n)) == 0
    assert 12 * 32768 + 16384 < n.value <= 12 * 32768 + 16384 + 256 * 8
    a = _args(half=1)
    assert f(ctypes.byref(a), ctypes.byref(n)) == 0
    assert lib.sparge_orthogonalize(ctypes.byref(a), FAKE, n.value - 1, None) == WS
    assert lib.sparge_orthogonalize(ctypes.byref(a), FAKE + 8, n.value, None) == MIS
    # 64 at a time
    for count, batch in ((64, 64), (65, 64), (200, 64)):
        assert f(ctypes.byref(_args(({},) * count, half=1)), ctypes.byref(n)) == 0
        assert batch * one < n.value <= batch * (one + 256 * 8)


def test_cpu_tensors_are_refused():
    x = torch.zeros(8, 8)
    with pytest.raises(ValueError):
        B.sparge_orthogonalize([x])
    with pytest.raises(ValueError):
        B.sparge_muon_step([x], [x], None, 0.1)
