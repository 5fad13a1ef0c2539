"""The log-sum-exp and the lengths among the tensors of a call that may share no memory, without
a GPU: what passes the checks ends at the missing workspace."""

import ctypes

import pytest

from block_sparse_attention_sparge_gb300 import binding as B
from test_cross_host import FAKE, INV, WS, _args

# (a forward that needs a workspace: one query over many keys)
FEW = dict(N=1, M=5000)
Q, K, V, O, DO, DQ, DK, DV = (FAKE << i for i in range(1, 9))
LSE = 2 * 4 * 4  # bytes of [2, 4, 1]


@pytest.fixture(scope="module")
def lib():
    return B.load_library(build_if_missing=True)


@pytest.mark.parametrize("kw,code", [
    (dict(lse=0), WS), (dict(lse=Q), INV), (dict(lse=K + 4), INV), (dict(lse=V - LSE + 4), INV),
    (dict(lse=V - LSE), WS), (dict(lse=O), INV), (dict(lse=O + 2 * 4 * 64 * 2 - 4), INV),
    (dict(lse=O + 2 * 4 * 64 * 2), WS), (dict(kv_len=FAKE), INV), (dict(kv_len=FAKE + LSE - 4), INV),
    (dict(kv_len=FAKE + LSE), WS), (dict(kv_len=FAKE - 8), WS), (dict(kv_len=O + 16), INV),
    (dict(kv_len=Q), WS), (dict(lse=DQ), WS),
])
def test_forward(lib, kw, code):
    assert lib.sparge_cross_fwd(ctypes.byref(_args(**FEW, **kw)), None, 0, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(), WS), (dict(lse=Q), WS), (dict(lse=DQ), INV), (dict(lse=DK + 64), INV),
    (dict(lse=DV - 4), INV), (dict(lse=DV - LSE), WS), (dict(kv_len=DQ), INV),
    (dict(kv_len=DK + 1024), INV), (dict(kv_len=DV - 4), INV), (dict(kv_len=DV - 8), WS),
])
def test_backward(lib, kw, code):
    assert lib.sparge_cross_bwd(ctypes.byref(_args(**FEW, **kw)), None, 0, None) == code
