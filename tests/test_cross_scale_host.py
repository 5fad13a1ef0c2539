"""Scales at fp32's end: the kernels take exponents to base 2, so scale * log2(e) has to be
finite too (else products of 0 become NaN)."""

import ctypes

import pytest

from block_sparse_attention_sparge_gb300 import binding as B
from test_cross_host import INV, WS, _args


@pytest.mark.parametrize("scale,code", [(2.3e38, WS), (-2.3e38, WS), (2.4e38, INV), (-3.4e38, INV),
                                        (1e-45, WS)])
def test_scales(scale, code):
    lib = B.load_library(build_if_missing=True)
    a, n = _args(N=1, M=5000, softmax_scale=scale), ctypes.c_size_t(0)
    assert lib.sparge_cross_fwd(ctypes.byref(a), None, 0, None) == code
    assert lib.sparge_cross_bwd(ctypes.byref(a), None, 0, None) == code
    fine = lib.sparge_cross_fwd_workspace_bytes(ctypes.byref(a), ctypes.byref(n))
    assert fine == (0 if code == WS else INV)
