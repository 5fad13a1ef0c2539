"""Where the outputs of the head layout may lie: the library's check against
every byte counted, over small layouts.  The calls stop before the device: those
that pass the check have no workspace."""

import ctypes
import random

import pytest

from block_sparse_attention_sparge_gb300 import binding as B

FAKE = 1 << 20  # never dereferenced


def _bytes(at, shape, stride, size):
    (b, n, h), d = shape, 64
    runs = [at + size * (i * stride[0] + j * stride[1] + k * stride[2])
            for i in range(b) for j in range(n) for k in range(h)]
    return [r + o for r in runs for o in range(0, d * size, 16)]


def _call(parts, b, n, f32):
    a = B.Heads()
    a.B, a.N, a.d, a.n_parts, a.x_type, a.norm, a.eps = b, n, 64, len(parts), f32, 1, 1e-6
    for i, (at, h, stride) in enumerate(parts):
        p = a.part[i]
        p.x = p.y = FAKE << (8 + i)
        p.x_stride = (n * h * 64, h * 64, 64)
        p.dx, p.dx_stride, p.H, p.dweight = at, tuple(stride), h, FAKE << 12
    return B.load_library().sparge_heads_bwd(ctypes.byref(a), None, 0, None)


def _strides(rng, shape):
    """Rows of one buffer in some order with gaps or overlaps."""
    order = rng.sample(range(3), 3)
    stride, reach = [0, 0, 0], 64
    for k in order:
        stride[k] = rng.choice([reach, reach, reach + 8 * rng.randint(0, 20),
                                8 * rng.randint(0, reach // 8 + 2)])
        reach = max(reach, stride[k] * shape[k])
    return stride


@pytest.mark.parametrize("seed", range(8))
def test_overlaps_against_every_byte(seed):
    rng = random.Random(seed)
    seen = set()
    for _ in range(400):
        f32 = rng.random() < 0.5
        size = 4 if f32 else 2
        b, n, h = (rng.randint(1, 3) for _ in range(3))
        stride = _strides(rng, (b, n, h))
        one = (FAKE, h, stride)
        own = _bytes(FAKE, (b, n, h), stride, size)
        # (one run repeated at size 1 is no repetition)
        bad = len(set(own)) < len(own)
        code = _call([one], b, n, f32)
        assert code == (B.SPARGE_ERR_INVALID_ARG if bad else B.SPARGE_ERR_WORKSPACE), (b, n, one)
        if bad:
            continue
        h2 = rng.choice([h, rng.randint(1, 3)])
        stride2 = rng.choice([stride, stride, _strides(rng, (b, n, h2))])
        at2 = FAKE + 16 * rng.choice([rng.randint(-30, 30), rng.randint(-300, 300),
                                      64 * size * rng.randint(-8, 8) // 16])
        other = _bytes(at2, (b, n, h2), stride2, size)
        bad = len(set(other)) < len(other) or bool(set(own) & set(other))
        code = _call([one, (at2, h2, stride2)], b, n, f32)
        assert code == (B.SPARGE_ERR_INVALID_ARG if bad else B.SPARGE_ERR_WORKSPACE), \
            (b, n, one, at2 - FAKE, h2, stride2)
        seen.add(bad)
    assert seen == {False, True}


def test_large_layouts_and_strides_past_any_memory():
    n, h = 200001, 12
    row = 3 * h * 64
    parts = [(FAKE + 2 * i * h * 64, h, (n * row, row, 64)) for i in range(3)]
    assert _call(parts, 2, n, False) == B.SPARGE_ERR_WORKSPACE
    late = [*parts[:2], (parts[2][0] - 16, *parts[2][1:])]
    assert _call(late, 2, n, False) == B.SPARGE_ERR_INVALID_ARG
    assert _call([(FAKE, 1, (1 << 40, 1 << 60, 64))], 1, 20, False) == B.SPARGE_ERR_INVALID_ARG
    # a stride that is not used may hold anything
    assert _call([(FAKE, 1, (1 << 60, 64, 1 << 61))], 1, 20, False) == B.SPARGE_ERR_WORKSPACE


def test_an_output_over_an_input_is_refused():
    a = B.Heads()
    a.B, a.N, a.d, a.n_parts, a.eps = 2, 100, 64, 1, 1e-6
    p = a.part[0]
    p.H, p.x, p.y, p.dx = 4, FAKE, FAKE + 2 * 25600, 1 << 40
    p.x_stride = p.dx_stride = (25600, 256, 64)
    lib = B.load_library()
    assert lib.sparge_heads_fwd(ctypes.byref(a), None) == B.SPARGE_ERR_INVALID_ARG
    p.dx = p.y + 16
    assert lib.sparge_heads_bwd(ctypes.byref(a), None, 0, None) == B.SPARGE_ERR_INVALID_ARG
    p.dx, a.norm = FAKE + 16, 1  # beside its input
    assert lib.sparge_heads_bwd(ctypes.byref(a), None, 0, None) == B.SPARGE_ERR_INVALID_ARG
