"""Argument checks of the attention over a context that need no GPU: every call
below fails validation before it reaches the device."""

import ctypes

import pytest
import torch

from block_sparse_attention_sparge_gb300 import binding as B

FAKE, ODD = 1 << 20, (1 << 20) + 8  # never dereferenced
INV, UNS, MIS = B.SPARGE_ERR_INVALID_ARG, B.SPARGE_ERR_UNSUPPORTED, B.SPARGE_ERR_MISALIGNED
WS = B.SPARGE_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    return B.load_library(build_if_missing=True)


def _args(**kw):
    a = B.Cross()
    a.B, a.Bk, a.H, a.Hk, a.N, a.M, a.d = 2, 2, 4, 2, 100, 50, 64
    for k, v in kw.items():
        if not k.endswith("_stride") and not isinstance(v, (tuple, list)):
            setattr(a, k, v)
    for i, n in enumerate(("q", "k", "v", "o", "dout", "dq", "dk", "dv")):
        keys = n in ("k", "v", "dk", "dv")
        heads, tokens = (a.Hk, a.M) if keys else (a.H, a.N)
        setattr(a, n, kw.get(n, FAKE << (i + 1)))
        stride = kw.get(n + "_stride", (heads * tokens * a.d, tokens * a.d, a.d))
        setattr(a, n + "_stride", (ctypes.c_int64 * 3)(*stride))
    a.lse = kw.get("lse", FAKE)
    return a


def test_struct_matches_the_header():
    assert ctypes.sizeof(B.Cross) == 312 == B._CROSS.size


BOTH = [
    (dict(B=0), INV), (dict(H=0), INV), (dict(Hk=0), INV), (dict(N=0), INV), (dict(M=0), INV),
    (dict(Hk=3), INV), (dict(Hk=8), INV), (dict(Bk=3), INV), (dict(B=3), INV), (dict(d=0), INV),
    (dict(d=80), UNS), (dict(d=256), UNS), (dict(N=600000), UNS), (dict(M=600000), UNS),
    (dict(softmax_scale=float("nan")), INV), (dict(softmax_scale=float("inf")), INV),
    (dict(B=1 << 21, Bk=1), UNS),
    (dict(q=0), INV), (dict(q=ODD), MIS), (dict(k=ODD), MIS), (dict(v=0), INV), (dict(o=0), INV),
    (dict(o=ODD), MIS), (dict(kv_len=FAKE + 2), MIS), (dict(lse=FAKE + 1), MIS),
    (dict(status=FAKE + 3), MIS),
    (dict(q_stride=(25600, 6400, 60)), MIS), (dict(q_stride=(25600, 0, 64)), INV),
    (dict(k_stride=(6400, -3200, 64)), INV), (dict(v_stride=(1 << 40, 3200, 64)), UNS),
]


@pytest.mark.parametrize("kw,code", BOTH)
def test_checks_of_both_directions(lib, kw, code):
    a = _args(**kw)
    n = ctypes.c_size_t(0)
    assert lib.sparge_cross_fwd(ctypes.byref(a), None, 0, None) == code
    assert lib.sparge_cross_bwd(ctypes.byref(a), None, 0, None) == code
    if set(kw) <= {"B", "Bk", "H", "Hk", "N", "M", "d", "softmax_scale"}:
        for f in (lib.sparge_cross_fwd_workspace_bytes, lib.sparge_cross_bwd_workspace_bytes):
            assert f(ctypes.byref(a), ctypes.byref(n)) == code


def test_checks_of_the_backward_and_workspaces(lib):
    n = ctypes.c_size_t(0)
    for kw, code in ((dict(lse=0), INV), (dict(dout=0), INV), (dict(dout=ODD), MIS),
                     (dict(dq=0), INV), (dict(dk=ODD), MIS), (dict(dv=0), INV),
                     (dict(dk_stride=(6400, 3200, 32)), INV),  # rows that overlap
                     (dict(), WS)):
        assert lib.sparge_cross_bwd(ctypes.byref(_args(**kw)), None, 0, None) == code, kw
    a = _args()
    assert lib.sparge_cross_fwd_workspace_bytes(ctypes.byref(a), ctypes.byref(n)) == 0
    assert n.value == 0  # few keys: one part
    assert lib.sparge_cross_bwd_workspace_bytes(ctypes.byref(a), ctypes.byref(n)) == 0
    assert n.value >= 2 * 4 * 100 * 4
    assert lib.sparge_cross_bwd(ctypes.byref(a), FAKE, n.value - 1, None) == WS
    assert lib.sparge_cross_bwd(ctypes.byref(a), ODD, n.value, None) == MIS
    a = _args(N=1, M=5000)
    assert lib.sparge_cross_fwd_workspace_bytes(ctypes.byref(a), ctypes.byref(n)) == 0
    assert n.value > 0
    assert lib.sparge_cross_fwd(ctypes.byref(a), None, 0, None) == WS
    assert lib.sparge_cross_fwd(ctypes.byref(a), ODD, n.value, None) == MIS
    assert lib.sparge_cross_fwd(None, None, 0, None) == INV
    assert lib.sparge_cross_fwd_workspace_bytes(ctypes.byref(a), None) == INV
    assert lib.sparge_cross_bwd_workspace_bytes(None, ctypes.byref(n)) == INV


def test_outputs_that_share_memory_are_refused(lib):
    q = FAKE << 1
    for kw in (dict(o=q), dict(o=q + 16), dict(o=(FAKE << 2) + 64), dict(o=FAKE << 3),
               dict(o_stride=(25600, 6400, 0))):
        assert lib.sparge_cross_fwd(ctypes.byref(_args(**kw)), None, 0, None) == INV, kw
    for kw in (dict(dq=q), dict(dk=FAKE << 2), dict(dv=FAKE << 7), dict(dq=FAKE << 5),
               dict(dq=FAKE << 4), dict(dv=(FAKE << 7) + 128)):
        assert lib.sparge_cross_bwd(ctypes.byref(_args(**kw)), None, 0, None) == INV, kw
    # slices of one buffer [2, 50, 2 (k, v), 2, 64] lie beside one another
    step = (50 * 256, 64, 256)
    a = _args(dk_stride=step, dv_stride=step, dv=(FAKE << 7) + 256)
    assert lib.sparge_cross_bwd(ctypes.byref(a), None, 0, None) == WS
    # strides of dimensions of size 1 are not used
    a = _args(B=1, Bk=1, q_stride=(3, 6400, 64), dk_stride=(-1, 3200, 64))
    assert lib.sparge_cross_bwd(ctypes.byref(a), None, 0, None) == WS


def test_cpu_tensors_are_refused():
    q = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.sparge_cross_fwd(q, q, q)
    with pytest.raises(ValueError):
        B.sparge_cross_bwd(q, q, q, q, torch.zeros(1, 2, 8), q)
