"""Calls of one kernel from two host threads, each with its own stream and
tensors and a row width of its own: every call succeeds, and gives the bits it
gives alone.  The loops call the C entry points with arguments made once, so
that the two are in the library at the same time as often as can be."""

import ctypes
import threading

import pytest
import torch

from block_sparse_attention_sparge_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
CALLS, AT_ONCE = 20000, 500  # calls of each thread, and between two waits


def _rand(seed, *shape, dtype=BF):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DEV, dtype)


def _recorded(call):
    """The C call that ``call`` makes, without its stream; what it returns."""
    made = []
    plain = B._call

    def record(fn, where, index, *args):
        made.append((fn, args))
        plain(fn, where, index, *args)

    B._call = record
    try:
        out = call()
    finally:
        B._call = plain
    (fn, args), = made
    return (lambda stream: fn(*args, stream)), out


def _heads_fwd(c):
    q, k, v = (_rand(i, 1, 8, c // 128, 128) for i in range(3))
    fn, out = _recorded(lambda: B.sparge_heads_fwd(q, k, v, norm="token"))
    return fn, out, (q, k, v)


def _heads_bwd(c):
    q, k = (_rand(i, 1, 8, c // 128, 128) for i in range(2))
    grads = [_rand(5 + i, 1, c // 128, 8, 128) for i in range(3)]
    fn, out = _recorded(lambda: B.sparge_heads_bwd(*grads, q, k, norm="head"))
    return fn, out[:3], (q, k, grads)


def _resnorm_fwd(c):
    x, b = _rand(1, 8, c, dtype=F32), _rand(2, 8, c)
    fn, out = _recorded(lambda: B.sparge_resnorm_fwd(x, b))
    return fn, out[:2], (x, b, out)


def _resnorm_bwd(c):
    x, b, dy, dh = (_rand(i, 8, c, dtype=t) for i, t in enumerate((F32, BF, F32, BF)))
    stats = B.sparge_resnorm_fwd(x, b)[2]
    fn, out = _recorded(lambda: B.sparge_resnorm_bwd(dy, dh, x, b, stats=stats))
    return fn, out[:2], (x, b, dy, dh, stats)


def _mask(n):
    """Above 512 kv-blocks: the selection that keeps its rows in shared memory."""
    q, k = _rand(1, 1, 1, n, 64), _rand(2, 1, 1, n, 64)
    shp, size = B._shape(q), ctypes.c_size_t(0)
    lib = B.load_library()
    assert lib.sparge_mask_workspace_bytes(ctypes.byref(shp), ctypes.byref(size)) == 0
    ws = torch.empty(size.value, dtype=torch.uint8, device=DEV)
    res = B.sparge_mask(q, k, 0.05, 0.5, want_csc=False, workspace=ws)
    args = [ctypes.byref(shp), B._ptr(q), B._ptr(k), 0.05, 0.5, 0.0, B._ptr(res["bitmask"]),
            B._ptr(res["row_idx"]), B._ptr(res["row_cnt"]), None, None, None, None, B._ptr(ws),
            ws.numel(), None]
    return (lambda st: lib.sparge_mask(*args, st)), [res["bitmask"]], (q, k, ws, res, shp)


def _mask_from_prob(n):
    mq, mk = B.num_blocks(n, 128), B.num_blocks(n, 64)
    prob = torch.softmax(_rand(1, 1, 1, mq, mk, dtype=F32), -1)
    res = B.sparge_mask_from_prob(prob, 0.05, 0.5, n, 64, want_csc=False)
    lib, shp = B.load_library(), B.Shape(1, 1, n, 64, 128, 64)
    args = [ctypes.byref(shp), B._ptr(prob), 0.05, 0.5, B._ptr(res["bitmask"]),
            B._ptr(res["row_idx"]), B._ptr(res["row_cnt"]), None, None]
    return (lambda st: lib.sparge_mask_from_prob(*args, st)), [res["bitmask"]], (prob, res, shp)


def _run(*made):
    torch.cuda.synchronize()
    want = [[t.clone() for t in out] for _, out, _ in made]
    refused, start = [0, 0], threading.Barrier(2)
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()

    def loop(i):
        fn, stream = made[i][0], streams[i]
        raw = ctypes.c_void_p(stream.cuda_stream)
        torch.cuda.set_device(stream.device)
        start.wait()
        for _ in range(CALLS // AT_ONCE):
            for _ in range(AT_ONCE):
                refused[i] += fn(raw) != 0
            stream.synchronize()

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert refused == [0, 0]
    for (_, out, _), ref in zip(made, want):
        assert all(torch.equal(a, b) for a, b in zip(out, ref))


@pytest.mark.parametrize("make", [_heads_fwd, _heads_bwd, _resnorm_fwd, _resnorm_bwd],
                         ids=lambda f: f.__name__)
@pytest.mark.parametrize("narrow,wide", [(1024, 1536), (2560, 5120)])
def test_two_widths_at_once(make, narrow, wide):
    _run(make(narrow), make(wide))


@pytest.mark.parametrize("make", [_mask, _mask_from_prob], ids=lambda f: f.__name__)
def test_two_lengths_of_the_mask_at_once(make):
    """528 and 1024 kv-blocks: rows of different size beside one another."""
    _run(make(33792), make(65536))
