"""Residual join and norm (sparge_resnorm_fwd / _bwd) against the 64-bit form."""

import pytest
import torch

import block_reference as R
from block_sparse_attention_sparge_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def _rand(g, *shape, dtype=F32, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g) * std + mean).to(dtype)


def _dev(t):
    return None if t is None else t.to(DEV)


class Case:
    """Inputs of one call; ``frames`` None: no modulation, 0: rows of [C]."""

    def __init__(self, b, n, c, tx, tb, norm, frames, post=False, branch=True, unit=True, seed=0,
                 offset=0.5):
        g = torch.Generator().manual_seed(seed)
        self.norm, self.unit = norm, unit
        self.x = _rand(g, b, n, c, dtype=tx, std=1.5, mean=offset)
        self.b = _rand(g, b, n, c, dtype=tb) if branch else None
        self.mods = {}
        if frames is not None:
            names = (["gate"] if branch else []) + (["scale", "shift"] if norm else [])
            if frames == 0:
                for name in names:
                    self.mods[name] = _rand(g, c, std=0.4, mean=0.1)
            else:
                table = _rand(g, b, frames, 3, c, std=0.4)  # rows 3 c apart
                for i, name in enumerate(names):
                    self.mods[name] = table[:, :, i]
        self.post = _rand(g, c, std=0.3, mean=1.0) if post else None
        self.dy, self.dh = _rand(g, b, n, c, dtype=tx), _rand(g, b, n, c, dtype=tb)

    def reference(self):
        return R.Resnorm(R.f64(self.x), R.f64(self.b), norm=self.norm, unit=self.unit,
                         post=R.f64(self.post), **{k: R.f64(v) for k, v in self.mods.items()})

    def forward(self, **more):
        mods = {k: self._mod(v) for k, v in self.mods.items()}
        return B.sparge_resnorm_fwd(_dev(self.x), _dev(self.b), norm=self.norm,
                                    unit_offset=self.unit, post_weight=_dev(self.post), **mods,
                                    **more)

    @staticmethod
    def _mod(v):
        if v.dim() == 1 or v.is_contiguous():
            return v.to(DEV)
        b, f, c = v.shape  # keep the strides of a slice
        table = torch.zeros(b, f, 3, c, device=DEV)
        table[:, :, 1] = v
        return table[:, :, 1]

    def backward(self, stats, dy=True, dh=True, **more):
        mods = {k: self._mod(v) for k, v in self.mods.items()}
        got = B.sparge_resnorm_bwd(_dev(self.dy) if dy else None, _dev(self.dh) if dh else None,
                                   _dev(self.x), _dev(self.b), stats=stats, norm=self.norm,
                                   unit_offset=self.unit, post_weight=_dev(self.post), **mods,
                                   **more)
        return dict(zip(("dx", "dbranch", "dgate", "dscale", "dshift", "dpost"), got))

    def check(self):
        ref = self.reference()
        y, h, stats = self.forward()
        if self.b is not None:
            R.check(y, ref.y, ref.y_bound(), "y")
            assert y.dtype == self.x.dtype
        if self.norm:
            R.check(h, ref.h, ref.h_bound(), "h")
        dh = self.dh if self.norm else None
        got = self.backward(stats, dh=self.norm is not None)
        self.check_grads(ref, got, self.dy, dh)
        again = self.backward(stats, dh=self.norm is not None)
        for k in got:
            assert got[k] is None or torch.equal(got[k], again[k]), k
        return ref, got

    def check_grads(self, ref, got, dy, dh):
        want = ref.backward(R.f64(dy), R.f64(dh))
        assert {k for k in got if got[k] is not None} == set(want)
        for k, (value, bound) in want.items():
            R.check(got[k], value, bound, k)


TYPES = [(BF, BF), (F32, BF), (F32, F32)]


@pytest.mark.parametrize("tx,tb", TYPES)
@pytest.mark.parametrize("norm", ["layer", "rms"])
@pytest.mark.parametrize("b,n,c,frames", [
    (1, 1, 8, 1), (2, 33, 128, 1), (1, 5, 264, 0), (3, 12, 1000, 4), (1, 7, 1536, 7),
    (2, 30, 64, 30), (1, 100, 1536, 1), (1, 9, 5120, 3), (2, 5, 8192, 1), (1, 3, 2056, None),
])
def test_forward_and_backward(b, n, c, frames, norm, tx, tb):
    Case(b, n, c, tx, tb, norm, frames).check()


@pytest.mark.parametrize("tx,tb", TYPES)
@pytest.mark.parametrize("norm", [None, "layer", "rms"])
@pytest.mark.parametrize("b,n,c,frames", [(2, 21, 256, 3), (1, 13, 1536, 0), (1, 4, 5120, 1)])
def test_norm_of_the_branch(b, n, c, frames, norm, tx, tb):
    Case(b, n, c, tx, tb, norm, frames, post=True).check()


@pytest.mark.parametrize("tx,tb", TYPES)
def test_norm_alone_and_join_alone(tx, tb):
    Case(2, 17, 320, tx, tb, "layer", 1, branch=False).check()
    Case(2, 17, 320, tx, tb, "rms", 0, branch=False, unit=False).check()
    Case(2, 17, 320, tx, tb, None, 17).check()
    case = Case(2, 17, 320, tx, tb, "layer", None, branch=False)
    y, h, _ = case.forward(h_dtype=tb)
    assert y.dtype == tx and h.dtype == tb


@pytest.mark.parametrize("unit", [True, False])
def test_weight_and_bias_of_the_model_beside_a_gate_for_each_sample(unit):
    """One row of scale and shift, one gate a frame: sums of both kinds."""
    case = Case(2, 24, 384, F32, BF, "layer", 3, unit=unit, post=True)
    g = torch.Generator().manual_seed(3)
    case.mods["scale"], case.mods["shift"] = _rand(g, 384, mean=1.0), _rand(g, 384)
    case.check()
    case.mods["gate"] = _rand(g, 1, 1, 384)  # one row for two samples
    case.check()


@pytest.mark.parametrize("b,n,c,frames", [(1, 9000, 64, 1), (1, 4096, 512, 2), (2, 3000, 1536, 1),
                                          (1, 3001, 2560, 1), (1, 700, 5120, 1)])
@pytest.mark.parametrize("tx,tb", [(BF, BF), (F32, F32)])
def test_sums_over_many_rows(b, n, c, frames, tx, tb):
    Case(b, n, c, tx, tb, "layer", frames, post=True, seed=1).check()


def test_only_one_of_the_two_gradients():
    case = Case(2, 11, 512, F32, BF, "layer", 1, post=True)
    ref = case.reference()
    stats = case.forward()[2]
    case.check_grads(ref, case.backward(stats, dy=False), None, case.dh)
    got = case.backward(stats, dh=False)
    case.check_grads(ref, got, case.dy, None)
    assert torch.equal(got["dx"].cpu(), case.dy)
    assert (got["dscale"] == 0).all() and (got["dshift"] == 0).all()
    got = case.backward(stats, want_mods=False)
    assert got["dgate"] is got["dscale"] is got["dshift"] is got["dpost"] is None
    # infinities in a row whose h has no gradient stay out of dx
    case.x[0, 3, 5] = float("inf")
    got = case.backward(stats, dh=False)
    assert torch.equal(got["dx"].cpu(), case.dy)


@pytest.mark.parametrize("c", [200, 1536])
def test_mean_far_above_the_spread(c):
    """Rows around 1000 with a spread of 1: the bound carries rstd * |y|, 2^10
    roundings; a variance from E[y^2] - E[y]^2 would be off by 2^20 of them."""
    case = Case(1, 14, c, F32, F32, "layer", None, branch=False, offset=1000.0)
    case.check()


def test_constant_rows_zero_rows_and_rows_of_infinities():
    case = Case(1, 9, 256, F32, F32, "layer", 1)
    case.x[0, 0], case.b[0, 0] = 3.0, 0.0       # deviation 0: z = 0
    case.x[0, 1], case.b[0, 1] = 0.0, 0.0
    clean = case.reference()
    _, h, stats = case.forward()
    R.check(h, clean.h, clean.h_bound())
    assert torch.equal(h[0, 0].cpu(), case.mods["shift"][0, 0])
    assert float(stats[1, 0].cpu()) == pytest.approx(1e3, rel=1e-6)
    case.x[0, 4, 9] = float("inf")
    case.b[0, 7, 0] = float("nan")
    y, h, _ = case.forward()
    keep = [0, 1, 2, 3, 5, 6, 8]
    R.check(h[:, keep], clean.h[:, keep], clean.h_bound()[:, keep])
    R.check(y[:, keep], clean.y[:, keep], clean.y_bound()[:, keep])
    assert h[0, 4].isnan().all() and h[0, 7].isnan().all() and y[0, 7, 0].isnan()


def test_against_differences():
    """Along a random direction of all inputs at once; the step 2^-10 leaves a
    third-order error below 2^-18 of the terms."""
    case = Case(2, 8, 72, F32, F32, "layer", 2, post=True, seed=5)
    _, _, stats = case.forward()
    got = case.backward(stats)
    ref = case.reference()
    bounds = {k: v[1] for k, v in ref.backward(R.f64(case.dy), R.f64(case.dh)).items()}
    ins = {"dx": case.x, "dbranch": case.b, "dgate": case.mods["gate"],
           "dscale": case.mods["scale"], "dshift": case.mods["shift"], "dpost": case.post}
    g = torch.Generator().manual_seed(6)
    for k, t in ins.items():
        v = torch.randn(t.shape, generator=g, dtype=torch.float64)

        def loss(e):
            p = {n: R.f64(a) + (e * v if n == k else 0) for n, a in ins.items()}
            r = R.Resnorm(p["dx"], p["dbranch"], p["dgate"], p["dscale"], p["dshift"], "layer",
                          True, p["dpost"])
            return float((r.y * R.f64(case.dy)).sum() + (r.h * R.f64(case.dh)).sum())

        e = 2.0 ** -10
        diff = (loss(e) - loss(-e)) / (2 * e)
        dot = float((R.f64(got[k]) * v).sum())
        room = float((bounds[k] * v.abs()).sum()) + 2.0 ** -18 * float((R.f64(got[k]) * v).abs().sum())
        assert abs(dot - diff) <= room, (k, dot, diff, room)


def test_two_dimensional_input_and_captured_replays():
    g = torch.Generator().manual_seed(8)
    x, b = _rand(g, 301, 1536).to(DEV), _rand(g, 301, 1536, dtype=BF).to(DEV)
    gate = _rand(g, 1, 7, 1536).to(DEV)
    scale, shift = _rand(g, 1, 7, 1536).to(DEV), _rand(g, 1, 7, 1536).to(DEV)
    dy, dh = _rand(g, 301, 1536).to(DEV), _rand(g, 301, 1536, dtype=BF).to(DEV)

    def both():
        y, h, st = B.sparge_resnorm_fwd(x, b, gate, scale, shift)
        return y, h, st, *B.sparge_resnorm_bwd(dy, dh, x, b, gate, scale, shift, st)[:5]

    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for seed in (9, 10):
        g = torch.Generator().manual_seed(seed)
        for t in (x, b, gate, scale, shift, dy, dh):
            t.copy_(_rand(g, *t.shape, dtype=t.dtype))
        graph.replay()
        torch.cuda.synchronize()
        want = both()
        for p, q in zip(got[:2] + got[3:], want[:2] + want[3:]):
            assert torch.equal(p, q)
        assert torch.equal(got[2][:2], want[2][:2])  # row 2 is not written without post_weight


def test_two_calls_at_once_on_two_streams():
    cases = [Case(1, 2000, 768, BF, BF, "rms", 1, post=True, seed=s) for s in (1, 2)]
    single = []
    for c in cases:
        st = c.forward()[2]
        single.append(c.backward(st))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for c, s in zip(cases, streams):
        with torch.cuda.stream(s):
            got.append(c.backward(c.forward()[2]))
    torch.cuda.synchronize()
    for p, q in zip(single, got):
        for k in p:
            assert p[k] is None or torch.equal(p[k], q[k])


def test_offsets_past_32_bits():
    n, c = 270001, 8192  # 2.2e9 elements
    x = torch.zeros((n, c), dtype=BF, device=DEV)
    assert x.numel() > 2 ** 31
    rows = [0, 262143, 262144, n - 1]
    g = torch.Generator().manual_seed(11)
    some = _rand(g, len(rows), c, dtype=BF)
    x[rows] = some.to(DEV)
    b = torch.zeros_like(x)
    b[rows] = some.to(DEV)
    gate = _rand(g, c).to(DEV)
    y, h, st = B.sparge_resnorm_fwd(x, b, gate)
    ref = R.Resnorm(R.f64(some)[None], R.f64(some)[None], gate=R.f64(gate))
    R.check(y[rows][None], ref.y, ref.y_bound())
    R.check(h[rows][None], ref.h, ref.h_bound())
    assert int(torch.count_nonzero(y.amax(1))) == len(rows)
    del y, h
    dx, db, dgate, *_ = B.sparge_resnorm_bwd(x, x, x, b, gate, stats=st)
    want = ref.backward(R.f64(some)[None], R.f64(some)[None])
    R.check(dx[rows][None], *want["dx"])
    R.check(db[rows][None], *want["dbranch"])
    # zero rows add nothing: the bound is that of a sum over the four rows
    R.check(dgate, *want["dgate"])


def test_refusals_on_the_device():
    x = torch.zeros(2, 6, 64, device=DEV)
    b = torch.zeros_like(x)
    m = torch.zeros(2, 1, 64, device=DEV)
    for bad in (dict(x=x.half()), dict(x=x[:, ::2]), dict(x=x.cpu()), dict(branch=b[:1]),
                dict(branch=b.half()), dict(norm="group"), dict(branch=b, gate=m.bfloat16()),
                dict(scale=m[:, :, ::2]), dict(scale=torch.zeros(2, 4, 64, device=DEV)),
                dict(scale=torch.zeros(1, 3, 64, device=DEV)),
                dict(scale=torch.zeros(3, 2, 64, device=DEV).transpose(0, 1)),
                dict(post_weight=torch.zeros(63, device=DEV)), dict(branch=b, h_dtype=BF)):
        with pytest.raises(ValueError):
            B.sparge_resnorm_fwd(**{"x": x, **bad})
    for bad, code in ((dict(norm=None), B.SPARGE_ERR_INVALID_ARG),
                      (dict(gate=m), B.SPARGE_ERR_INVALID_ARG),
                      (dict(branch=b, norm=None, scale=m), B.SPARGE_ERR_INVALID_ARG),
                      (dict(x=x.bfloat16(), branch=b), B.SPARGE_ERR_UNSUPPORTED),
                      (dict(x=x.bfloat16(), h_dtype=F32), B.SPARGE_ERR_UNSUPPORTED),
                      (dict(x=torch.zeros(1, 2, 60, device=DEV)), B.SPARGE_ERR_UNSUPPORTED),
                      (dict(x=torch.zeros(1, 2, 8200, device=DEV)), B.SPARGE_ERR_UNSUPPORTED),
                      (dict(x=torch.zeros(1, 0, 64, device=DEV)), B.SPARGE_ERR_INVALID_ARG),
                      (dict(eps=float("nan")), B.SPARGE_ERR_INVALID_ARG),
                      (dict(scale=m, shift=torch.zeros(2, 3, 64, device=DEV)),
                       B.SPARGE_ERR_UNSUPPORTED),
                      (dict(scale=torch.zeros(2, 65, device=DEV)[:, None, :64]),
                       B.SPARGE_ERR_MISALIGNED)):
        with pytest.raises(B.SpargeError) as e:
            B.sparge_resnorm_fwd(**{"x": x, **bad})
        assert e.value.code == code, bad
    st = torch.zeros(3, 12, device=DEV)
    for bad in (dict(dy=x.bfloat16(), dh=None), dict(dy=None, dh=x[:1]),
                dict(dy=x, dh=None, stats=st[:, :6])):
        with pytest.raises(ValueError):
            B.sparge_resnorm_bwd(**{"x": x, "stats": st, **bad})
    for bad in (dict(dy=None, dh=None), dict(dy=x, dh=x, stats=None),
                dict(dy=x, dh=x, branch=b, norm=None)):
        with pytest.raises(B.SpargeError) as e:
            B.sparge_resnorm_bwd(**{"x": x, "stats": st, **bad})
        assert e.value.code == B.SPARGE_ERR_INVALID_ARG
    with pytest.raises(B.SpargeError) as e:
        B.sparge_resnorm_bwd(x, x, x, scale=m, stats=st,
                             workspace=torch.empty(0, dtype=torch.uint8, device=DEV))
    assert e.value.code in (B.SPARGE_ERR_WORKSPACE,)
