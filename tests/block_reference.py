"""Plain 64-bit forms of the operators around the attention, from their
formulas, with bounds for what fp32 arithmetic may be off by.

Bounds: one fp32 operation is off by at most 2^-24 of its result.  The longest
chain of additions behind a row's sum is 8 channels of a thread, 5 steps in a
warp and 32 warps; with the handful of products around it every fp32 result is
within K = 64 * 2^-24 of the sum of the absolute values of its terms (128 for
the backward, which chains two such sums).  Rounding to bf16 adds 2^-8 of the
value."""

import math

import torch

U = 2.0 ** -24
K = 64 * U
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


def f64(t):
    return None if t is None else t.detach().cpu().double()


def check(got, ref, bound, what=""):
    """|got - ref| <= bound + half a step of got's type, everywhere."""
    g = f64(got)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    off = (g - ref).abs()
    # 2^-133: half of bf16's smallest step, for results that round to it
    lim = bound + HALF_STEP[got.dtype] * ref.abs() * (1 + K) + 2.0 ** -133
    bad = ~(off <= lim)
    if bad.any():
        i = int((off / lim).nan_to_num(math.inf).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off; worst at {i}: "
                             f"{g.flatten()[i]} against {ref.flatten()[i]}, "
                             f"bound {lim.flatten()[i]}")


# ------------------------------------------------------------------- heads
def positions(B, N, grid=None, pos=None):
    """int64 [B, N, 3]."""
    if pos is not None:
        return pos.cpu().long().expand(B, N, 3)
    out = torch.zeros(B, N, 3, dtype=torch.int64)
    for b, (t, h, w) in enumerate(grid.cpu().tolist()):
        if min(t, h, w) < 1:
            continue
        for n in range(min(N, t * h * w)):
            out[b, n] = torch.tensor([n // (h * w), n // w % h, n % w])
    return out


def angles(p, pairs, d, theta=10000.0, scale=(1.0, 1.0, 1.0)):
    """cos, sin [B, N, 1, d / 2]; the frequencies exactly as stated, the
    products reduced in 64 bits (positions below 2^31 lose 2^-21 turns)."""
    f, axis = torch.zeros(d // 2, dtype=torch.float64), torch.zeros(d // 2, dtype=torch.long)
    j = 0
    for a, n in enumerate(pairs):
        for i in range(n):
            f[j], axis[j] = scale[a] * theta ** (-i / n), a
            j += 1
    ang = p[..., axis].double() * f
    return ang.cos()[:, :, None], ang.sin()[:, :, None]


def turn(x, cos, sin, interleaved):
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else x.chunk(2, -1)
    u, v = a * cos - b * sin, a * sin + b * cos
    return torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)


def pair_size(x, interleaved):
    """|a| + |b| of each pair, at both of its places."""
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else x.chunk(2, -1)
    s = a.abs() + b.abs()
    return torch.stack([s, s], -1).flatten(-2) if interleaved else torch.cat([s, s], -1)


def heads_fwd(x, w, norm, cs, interleaved, eps=1e-6):
    """[B, H, N, d] in 64 bits, and its bound.  cs None: no rotation."""
    u = x
    if norm is not None:
        dims = (-2, -1) if norm == "token" else (-1,)
        u = x * (x.square().mean(dims, keepdim=True) + eps).rsqrt()
        if w is not None:
            u = u * (w.view(x.shape[2:]) if norm == "token" else w)
    y = turn(u, *cs, interleaved) if cs is not None else u
    bound = K * pair_size(u, interleaved)
    return y.transpose(1, 2), bound.transpose(1, 2)


def heads_bwd(dy, x, w, norm, cs, interleaved, eps=1e-6):
    """dx, its bound, dw, its bound."""
    dy = dy.transpose(1, 2)
    g = turn(dy, cs[0], -cs[1], interleaved) if cs is not None else dy
    size = pair_size(dy, interleaved)  # |g| and what its rounding goes by
    if norm is None:
        return g, 2 * K * size, None, None
    dims = (-2, -1) if norm == "token" else (-1,)
    r = (x.square().mean(dims, keepdim=True) + eps).rsqrt()
    xh = x * r
    wv = torch.ones_like(x) if w is None else (w.view(x.shape[2:]) if norm == "token" else w)
    q = g * wv
    dx = r * (q - xh * (q * xh).mean(dims, keepdim=True))
    sq = size * wv.abs()
    bound = 2 * K * r * (sq + xh.abs() * (sq * xh.abs()).mean(dims, keepdim=True))
    over = (0, 1) if norm == "token" else (0, 1, 2)
    terms = x.shape[0] * x.shape[1] * (1 if norm == "token" else x.shape[2])
    dw = (g * xh).sum(over).flatten()
    dwb = (2 * K + terms * U) * (size * xh.abs()).sum(over).flatten()
    return dx, bound, dw, dwb


# ----------------------------------------------------------------- resnorm
def rows_of(m, B, N):
    """[C] or [B, F, C] for every token, [B, N, C]."""
    if m.dim() == 1:
        return m.expand(B, N, -1)
    return m.expand(B, -1, -1).repeat_interleave(N // m.shape[1], 1)


def sum_to(t, m):
    if m.dim() == 1:
        return t.sum((0, 1))
    if m.shape[0] != t.shape[0]:
        t = t.sum(0, keepdim=True)
    return t.unflatten(1, (m.shape[1], -1)).sum(2)


class Resnorm:
    """The operator's intermediate values in 64 bits; x [B, N, C]."""

    def __init__(self, x, b=None, gate=None, scale=None, shift=None, norm="layer", unit=True,
                 post=None, eps=1e-6):
        B, N, C = x.shape
        self.__dict__.update(x=x, b=b, norm=norm, post=post)
        self.mods = dict(gate=gate, scale=scale, shift=shift, post=post)
        self.gate = rows_of(gate, B, N) if gate is not None else torch.ones_like(x)
        gain = rows_of(scale, B, N) if scale is not None else torch.ones_like(x)
        self.gain = gain + 1 if unit and scale is not None else gain
        self.shift = rows_of(shift, B, N) if shift is not None else torch.zeros_like(x)
        self.y, self.size = x, x.abs()
        if b is not None:
            self.rb = torch.ones(B, N, 1, dtype=torch.float64)
            n = b
            if post is not None:
                self.rb = (b.square().mean(-1, keepdim=True) + eps).rsqrt()
                n = b * self.rb * post
            self.n = n
            self.y = x + self.gate * n
            self.size = x.abs() + (self.gate * n).abs()
        if norm is not None:
            mean = self.y.mean(-1, keepdim=True) if norm == "layer" else 0.0 * self.y[..., :1]
            c = self.y - mean
            self.mean = mean
            self.rstd = (c.square().mean(-1, keepdim=True) + eps).rsqrt()
            self.z = c * self.rstd
            self.h = self.z * self.gain + self.shift
            # what the rounding of y does to z: its own part, the mean's, the
            # deviation's
            big = self.size.amax(-1, keepdim=True) * self.rstd
            self.z_bound = K * (1 + self.z.abs()) * (1 + big)

    def y_bound(self):
        return K * self.size

    def h_bound(self):
        return self.z_bound * self.gain.abs() + K * (self.shift.abs() + self.h.abs())

    def backward(self, dy, dh):
        """{name: (value, bound)}"""
        x, B, N = self.x, *self.x.shape[:2]
        zero = torch.zeros_like(x)
        dy = zero if dy is None else dy
        d, bd, out = dy, K * dy.abs(), {}
        grow = 2 * K + U * B * N
        if self.norm is not None:
            if dh is None:
                dh = zero
            g = dh * self.gain
            gm = g.mean(-1, keepdim=True) if self.norm == "layer" else 0.0 * g[..., :1]
            gz = (g * self.z).mean(-1, keepdim=True)
            d = dy + self.rstd * (g - gm - self.z * gz)
            ag = g.abs()
            am, az = ag.mean(-1, keepdim=True), (ag * self.z.abs()).mean(-1, keepdim=True)
            eg = (ag * self.z_bound).mean(-1, keepdim=True)  # z's bound in the mean
            bd = K * dy.abs() + self.rstd * (2 * K * (ag + am + self.z.abs() * az)
                                             + self.z_bound * az + self.z.abs() * eg)
            if self.mods["scale"] is not None:
                out["dscale"] = (sum_to(dh * self.z, self.mods["scale"]),
                                 sum_to(dh.abs() * (grow * self.z.abs() + self.z_bound),
                                        self.mods["scale"]))
            if self.mods["shift"] is not None:
                out["dshift"] = (sum_to(dh, self.mods["shift"]),
                                 grow * sum_to(dh.abs(), self.mods["shift"]))
        out["dx"] = (d, bd)
        if self.b is not None:
            if self.mods["gate"] is not None:
                out["dgate"] = (sum_to(d * self.n, self.mods["gate"]),
                                sum_to((grow * d.abs() + bd) * self.n.abs(), self.mods["gate"]))
            e, be = d * self.gate, (bd + K * d.abs()) * self.gate.abs()
            if self.post is not None:
                bh = self.b * self.rb
                out["dpost"] = ((e * bh).sum((0, 1)),
                                ((grow * e.abs() + be) * bh.abs()).sum((0, 1)))
                q, bq = e * self.post, (be + K * e.abs()) * self.post.abs()
                e = self.rb * (q - bh * (q * bh).mean(-1, keepdim=True))
                mean_q = ((q.abs() * 2 * K + bq) * bh.abs()).mean(-1, keepdim=True)
                be = self.rb * (bq + 2 * K * q.abs()
                                + bh.abs() * (mean_q + 2 * K * (q * bh).abs().mean(-1, keepdim=True)))
            out["dbranch"] = (e, be)
        return out
