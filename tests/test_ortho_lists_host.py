"""A list of both forms (fp16 values, fp16 pairs) is one list: its tensors are checked against
one another, without a GPU."""

import ctypes

import pytest

from block_sparse_attention_sparge_gb300 import binding as B
from test_ortho_host import FAKE, INV, UNS, _args


@pytest.fixture(scope="module")
def lib():
    return B.load_library(build_if_missing=True)


@pytest.mark.parametrize("rows,kw,code", [
    (({}, dict(out_type=0)), {}, 0),
    # a bf16 result on an fp32 gradient, a momentum and a result of either type
    ((dict(out_type=0, out=(FAKE << 4) + 65536), {}), {}, INV),
    ((dict(out_type=0, momentum=FAKE << 9), dict(momentum=(FAKE << 9) + 400)), {}, INV),
    ((dict(out_type=0, out=FAKE << 9), dict(out=(FAKE << 9) + 1196)), {}, INV),
    ((dict(out_type=0, out=FAKE << 9), dict(out=(FAKE << 9) + 1200)), {}, 0),
    ((dict(rows=0),), {}, INV), ((dict(rows=65537),), {}, UNS), (({},), dict(steps=-1), INV),
])
def test_check(lib, rows, kw, code):
    assert lib.sparge_orthogonalize_check(ctypes.byref(_args(rows, **kw))) == code


def test_check_of_nothing(lib):
    assert lib.sparge_orthogonalize_check(None) == INV
