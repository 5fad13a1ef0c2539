"""Cases of the operators around the sparse attention of a video transformer block.

* ``heads``: query, key and value projections [B, N, H, d] to the attention's
  bf16 [B, H, N, d]: RMS norm of Q and K, rotary positions with a time, a
  height and a width axis, the layout change and the cast; and its gradients.
* ``resnorm``: the residual join of one half-block and the norm of the next:
  y = x + gate * branch, h = norm(y) * (1 + scale) + shift; and its gradients.
* ``clip``: the global norm of a list of gradients and the clipped gradients.

``own = False`` computes them in elementary torch operations in 32 bits
(angles in 64), rounded once at the end; ``own = True`` calls the library.
"""

import functools
import math

import torch

own = False

EPS = 1e-6
THETA = 10000.0
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases
def _heads(name, way, B, grid, H, d, dtype, norm, interleaved, pad=0, far=0):
    """``pad`` tokens follow the largest sample's grid; sample b has b frames
    fewer.  ``far``: positions given per token, the frames counted from it."""
    return {"name": name, "op": "heads", "way": way, "B": B, "t": grid[0], "h": grid[1],
            "w": grid[2], "N": grid[0] * grid[1] * grid[2] + pad, "H": H, "d": d, "dtype": dtype,
            "norm": norm, "interleaved": interleaved, "far": far}


def _resnorm(name, way, B, frames, per, C, x, branch, norm, affine=False, post=False):
    """N = frames * per tokens; gate, scale and shift for each frame of a
    sample.  ``affine``: the norm has a weight and a bias of the model
    instead.  ``post``: the branch passes an RMS norm before its gate."""
    return {"name": name, "op": "resnorm", "way": way, "B": B, "N": frames * per,
            "frames": frames, "C": C, "x": x, "branch": branch, "norm": norm, "affine": affine,
            "post": post}


def _clip(name, layers, width, wide, dtype, max_norm):
    """Gradients of ``layers`` blocks: four square projections and, where
    ``wide`` > 0, biases, norm weights, a modulation table and an MLP."""
    return {"name": name, "op": "clip", "layers": layers, "width": width, "wide": wide,
            "dtype": dtype, "max_norm": max_norm}


def listed():
    return [
        # one small clip of a test model: latency
        _heads("heads_small_fwd", "fwd", 1, (4, 16, 16), 2, 64, "fp32", "head", False),
        # the 480p video shape, slices of one fused projection
        _heads("heads_480p_fwd", "fwd", 1, (21, 30, 52), 12, 128, "bf16", "token", True),
        _heads("heads_480p_bwd", "bwd", 1, (21, 30, 52), 12, 128, "bf16", "token", True),
        # the 720p video shape
        _heads("heads_720p_fwd", "fwd", 1, (21, 45, 80), 40, 128, "bf16", "token", True),
        # a padded batch of clips of different lengths, later chunks of long
        # videos (positions given), fp32 projections, odd head count
        _heads("heads_ragged_bwd", "bwd", 3, (9, 17, 31), 7, 64, "fp32", "head", False, 258, 40000),
        # a few tokens of a narrow test model: latency
        _resnorm("resnorm_small_fwd", "fwd", 2, 1, 33, 128, "fp32", "fp32", "layer"),
        # between two half-blocks at the 480p shape: fp32 residual stream
        _resnorm("resnorm_480p_fwd", "fwd", 1, 1, 32760, 1536, "fp32", "bf16", "layer"),
        _resnorm("resnorm_480p_bwd", "bwd", 1, 1, 32760, 1536, "fp32", "bf16", "layer"),
        # one modulation for each frame, norms before and after, bf16 stream
        _resnorm("resnorm_frames_bwd", "bwd", 1, 21, 1560, 1536, "bf16", "bf16", "rms", False, True),
        # the 720p shape, before the norm with a weight and a bias
        _resnorm("resnorm_720p_fwd", "fwd", 1, 1, 75600, 5120, "bf16", "bf16", "layer", True),
        # the four projections of a test block: latency
        _clip("clip_small", 1, 128, 0, "fp32", 1.0),
        # every gradient of a stack of blocks of the 480p width
        _clip("clip_stack", 24, 1536, 4, "bf16", 1.0),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    case = _draw(rng)
    del case["name"]
    return case


def _draw(rng):
    op = rng.choice(["heads", "resnorm", "clip"])
    way = rng.choice(["fwd", "bwd"])
    # values of one [B, N, C] tensor: no pass moves more than the largest listed one
    most = 180_000_000 if way == "fwd" else 90_000_000
    if op == "heads":
        d = rng.choice([64, 128])
        H = _spread(rng, 1, 40)
        B = rng.choice([1, 1, 2, 3])
        most //= B * H * d
        n = _spread(rng, 1, min(most, 131072))
        t = rng.randint(1, max(1, min(33, n)))
        h = max(1, min(n // t, _spread(rng, 1, 90)))
        w = max(1, n // (t * h))
        pad = rng.choice([0, 0, rng.randint(1, 300)])
        pad = max(0, min(pad, most - t * h * w))
        far = rng.choice([0, 0, rng.randint(1, 1000000)])
        return _heads("", way, B, (t, h, w), H, d, rng.choice(["bf16", "bf16", "fp32"]),
                      rng.choice(["token", "head", "none"]), rng.random() < 0.5, pad, far)
    if op == "resnorm":
        C = 8 * _spread(rng, 4, 1024)
        B = rng.choice([1, 1, 2, 3])
        most //= B * C
        n = _spread(rng, 1, min(most, 131072))
        frames = rng.choice([1, 1, rng.randint(1, 33), n])
        frames = max(1, min(frames, n))
        x = rng.choice(["bf16", "fp32"])
        branch = "bf16" if x == "bf16" else rng.choice(["bf16", "fp32"])
        return _resnorm("", way, B, frames, n // frames, C, x, branch,
                        rng.choice(["layer", "rms"]), rng.random() < 0.3, rng.random() < 0.3)
    width = _spread(rng, 5, 1536)
    return _clip("", rng.randint(1, 24), width, rng.choice([0, 2, 4]), rng.choice(["bf16", "fp32"]),
                 rng.choice([0.1, 1.0, 1e6]))


# ------------------------------------------------------------------ inputs
def _pairs(d):
    side = d // 6
    return (d // 2 - 2 * side, side, side)


def _clip_shapes(case):
    C = case["width"]
    one = [(C, C)] * 4
    if case["wide"]:
        wide = case["wide"] * C
        one += [(C,)] * 4 + [(C,), (C,), (6, C), (wide, C), (wide,), (C, wide), (C,)]
    return one * case["layers"]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape, dtype=torch.float32, std=1.0, mean=0.0):
        return torch.randn(shape, generator=gen, device="cuda").mul_(std).add_(mean).to(dtype)

    st = dict(case)
    if case["op"] == "heads":
        B, N, H, d = (case[k] for k in ("B", "N", "H", "d"))
        C, dtype = H * d, TYPES[case["dtype"]]
        # a projection's outputs: channels of different size
        qkv = (rand(B, N, 3 * C) * rand(3 * C).abs().add_(0.2)).to(dtype)
        st["q"], st["k"], st["v"] = (qkv[..., i * C:(i + 1) * C].unflatten(-1, (H, d))
                                     for i in range(3))
        width = {"token": C, "head": d, "none": 0}[case["norm"]]
        st["wq"], st["wk"] = ((rand(width, std=0.1, mean=1.0).to(dtype) if width else None)
                              for _ in range(2))
        grid = torch.tensor([[max(1, case["t"] - b), case["h"], case["w"]] for b in range(B)],
                            dtype=torch.int32)
        st["grid"], st["pos"] = grid.to("cuda"), None
        if case["far"]:
            # the positions of a clip that starts at a later frame; padding at 0
            n = torch.arange(N)
            per = grid[0, 1] * grid[0, 2]
            pos = torch.stack([n // per + case["far"], n // grid[0, 2] % grid[0, 1],
                               n % grid[0, 2]], -1)
            inside = n < (grid[:, 0] * per)[:, None]
            st["pos"] = (pos * inside[..., None]).to("cuda", torch.int32)
            st["grid"] = None
        if case["way"] == "bwd":
            st["dq"], st["dk"], st["dv"] = (rand(B, H, N, d, dtype=torch.bfloat16)
                                            for _ in range(3))
            st["dqkv"] = torch.empty(B, N, 3 * C, dtype=dtype, device="cuda")
        return st
    if case["op"] == "resnorm":
        B, N, C, F = (case[k] for k in ("B", "N", "C", "frames"))
        tx, tb = TYPES[case["x"]], TYPES[case["branch"]]
        # a residual stream: an offset and a size of its own in each channel
        st["x"] = (rand(B, N, C) * rand(C).abs().add_(0.5) + rand(C, std=0.5)).to(tx)
        st["b"] = rand(B, N, C, dtype=tb)
        table = rand(B, F, 6, C, std=0.3)
        st["shift"], st["scale"], st["gate"] = table[:, :, 0], table[:, :, 1], table[:, :, 2]
        if case["affine"]:
            st["scale"], st["shift"] = rand(C, std=0.1, mean=1.0), rand(C, std=0.1)
        st["post"] = rand(C, std=0.1, mean=1.0) if case["post"] else None
        if case["way"] == "bwd":
            st["dy"], st["dh"] = rand(B, N, C, dtype=tx), rand(B, N, C, dtype=tb)
            # what the forward left: mean and 1/deviation of y, of the branch
            b = st["b"].float()
            rb = torch.ones(B, N, device="cuda")
            if case["post"]:
                rb = (b.double().square().mean(-1) + EPS).rsqrt().float()
                b = b * rb[..., None] * st["post"]
            y = b.mul_(_rows(st["gate"], N)).add_(st["x"]).double()
            mean = y.mean(-1) if case["norm"] == "layer" else y.new_zeros(B, N)
            var = (y - mean[..., None]).square_().mean(-1)
            st["stats"] = torch.stack([mean.float(), (var + EPS).rsqrt().float(), rb])
        return st
    shapes, dtype = _clip_shapes(case), TYPES[case["dtype"]]
    st["grads"] = [rand(*s, dtype=dtype, std=2e-3) for s in shapes]
    sizes = [g.numel() for g in st["grads"]]
    places = [0]
    for n in sizes:
        places.append(places[-1] + (n + 7) // 8 * 8)  # 16-byte places in one buffer
    st["places"] = places
    st["flat"] = torch.zeros(places[-1], dtype=dtype, device="cuda")
    st["out"] = [st["flat"][p:p + n].view(s) for p, n, s in zip(places, sizes, shapes)]
    return st


# ---------------------------------------------------------------- plain form
def _rows(m, N):
    """[C] or [B, F, C] for each of N tokens."""
    if m.dim() == 1:
        return m
    return m.repeat_interleave(N // m.shape[1], dim=1)


def _frequencies(d):
    return torch.tensor([[THETA ** (-j / p), a] for a, p in enumerate(_pairs(d)) for j in range(p)],
                        dtype=torch.float64, device="cuda")


def _cos_sin(st):
    N = st["N"]
    pos = st["pos"]
    if pos is None:
        t, h, w = (st["grid"][:, i, None].long() for i in range(3))
        n = torch.arange(N, device="cuda")[None]
        pos = torch.stack([n // (h * w), n // w % h, n % w], -1) * (n < t * h * w)[..., None]
    f = _frequencies(st["d"])
    angle = pos[..., f[:, 1].long()].double() * f[:, 0]
    return angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]


def _rotate(x, cos, sin, interleaved):
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
    else:
        a, b = x.chunk(2, -1)
    u, v = a * cos - b * sin, a * sin + b * cos
    return torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)


def _mean(x, norm):
    return x.mean((-2, -1), keepdim=True) if norm == "token" else x.mean(-1, keepdim=True)


def _plain_heads(st):
    norm, shape = st["norm"], (st["B"], st["N"], st["H"], st["d"])
    cos, sin = _cos_sin(st)
    out = []
    for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        x = x.float()
        if norm != "none":
            w = w.float().view(shape[2:] if norm == "token" else shape[3:])
            x = x * (_mean(x.square(), norm) + EPS).rsqrt() * w
        out.append(_rotate(x, cos, sin, st["interleaved"]).to(torch.bfloat16)
                   .transpose(1, 2).contiguous())
    return {"q": out[0], "k": out[1],
            "v": st["v"].to(torch.bfloat16).transpose(1, 2).contiguous()}


def _plain_heads_bwd(st):
    norm, shape, dtype = st["norm"], (st["B"], st["N"], st["H"], st["d"]), TYPES[st["dtype"]]
    cos, sin = _cos_sin(st)
    grads, weights = [], []
    for dout, x, w in ((st["dq"], st["q"], st["wq"]), (st["dk"], st["k"], st["wk"])):
        g = _rotate(dout.float().transpose(1, 2), cos, -sin, st["interleaved"])
        if norm != "none":
            x = x.float()
            r = (_mean(x.square(), norm) + EPS).rsqrt()
            x = x * r
            dw = (g * x).sum((0, 1) if norm == "token" else (0, 1, 2))
            weights.append(dw.reshape(-1).to(w.dtype))
            g = g * w.float().view(shape[2:] if norm == "token" else shape[3:])
            g = r * (g - x * _mean(g * x, norm))
        grads.append(g.to(dtype).flatten(2))
    grads.append(st["dv"].to(dtype).transpose(1, 2).flatten(2))
    return {"dqkv": torch.cat(grads, -1), "dw": weights}


def _plain_resnorm(st):
    N = st["N"]
    x, b = st["x"].float(), st["b"].float()
    if st["post"] is not None:
        b = b * (b.square().mean(-1, keepdim=True) + EPS).rsqrt() * st["post"]
    y = x + _rows(st["gate"], N) * b
    z = y - y.mean(-1, keepdim=True) if st["norm"] == "layer" else y
    z = z * (z.square().mean(-1, keepdim=True) + EPS).rsqrt()
    gain = st["scale"] if st["affine"] else 1 + _rows(st["scale"], N)
    h = z * gain + _rows(st["shift"], N)
    return {"y": y.to(st["x"].dtype), "h": h.to(st["b"].dtype)}


def _over(t, m):
    """Sums of [B, N, C] over the tokens that share a row of ``m``."""
    if m.dim() == 1:
        return t.sum((0, 1))
    return t.unflatten(1, (m.shape[1], -1)).sum(2)


def _plain_resnorm_bwd(st):
    N = st["N"]
    x, b, dy, dh = (st[k].float() for k in ("x", "b", "dy", "dh"))
    mean, rstd, rb = (s[..., None] for s in st["stats"])
    gate = _rows(st["gate"], N)
    post = st["post"]
    bh = b * rb if post is not None else b
    n = bh * post if post is not None else b
    z = (x + gate * n - mean) * rstd
    g = dh * (st["scale"] if st["affine"] else 1 + _rows(st["scale"], N))
    g2 = g - z * (g * z).mean(-1, keepdim=True)
    if st["norm"] == "layer":
        g2 = g2 - g.mean(-1, keepdim=True)
    d = dy + rstd * g2
    out = {"dscale": _over(dh * z, st["scale"]), "dshift": _over(dh, st["shift"]),
           "dgate": _over(d * n, st["gate"])}
    db = d * gate
    if post is not None:
        out["dpost"] = (db * bh).sum((0, 1))
        db = db * post
        db = rb * (db - bh * (db * bh).mean(-1, keepdim=True))
    out["dx"], out["db"] = d.to(st["x"].dtype), db.to(st["b"].dtype)
    return out


def _plain_clip(st):
    norm = torch.stack([g.float().square().sum() for g in st["grads"]]).sum().sqrt()
    factor = (st["max_norm"] / (norm + EPS)).clamp(max=1.0)
    flat = torch.zeros_like(st["flat"])
    for g, p in zip(st["grads"], st["places"]):
        flat[p:p + g.numel()] = (g.float() * factor).flatten()
    return {"norm": norm, "grads": flat}


# --------------------------------------------------------------- the library
@functools.lru_cache(maxsize=None)
def _axes(d, interleaved):
    from block_sparse_attention_sparge_gb300 import RopeAxes
    return RopeAxes(d, _pairs(d), theta=THETA, interleaved=interleaved)


def _own(st):
    import block_sparse_attention_sparge_gb300 as S
    if st["op"] == "heads":
        norm = None if st["norm"] == "none" else st["norm"]
        how = dict(rope=_axes(st["d"], st["interleaved"]), grid=st["grid"], pos=st["pos"],
                   norm=norm, q_weight=st["wq"], k_weight=st["wk"], eps=EPS)
        if st["way"] == "fwd":
            q, k, v = S.sparge_heads_fwd(st["q"], st["k"], st["v"], **how)
            return {"q": q, "k": k, "v": v}
        out = [t.unflatten(-1, (st["H"], st["d"])) for t in st["dqkv"].chunk(3, -1)]
        got = S.sparge_heads_bwd(st["dq"], st["dk"], st["dv"], st["q"], st["k"], out=out, **how)
        return {"dqkv": st["dqkv"], "dw": [w for w in got[3:] if w is not None]}
    if st["op"] == "resnorm":
        how = dict(norm=st["norm"], unit_offset=not st["affine"], post_weight=st["post"])
        if st["way"] == "fwd":
            y, h, _ = S.sparge_resnorm_fwd(st["x"], st["b"], st["gate"], st["scale"], st["shift"],
                                           eps=EPS, **how)
            return {"y": y, "h": h}
        dx, db, dgate, dscale, dshift, dpost = S.sparge_resnorm_bwd(
            st["dy"], st["dh"], st["x"], st["b"], st["gate"], st["scale"], st["shift"],
            st["stats"], **how)
        out = {"dscale": dscale, "dshift": dshift, "dgate": dgate, "dx": dx, "db": db}
        return out | {"dpost": dpost} if dpost is not None else out
    return {"norm": S.sparge_clip_grads(st["grads"], st["max_norm"], out=st["out"], eps=EPS),
            "grads": st["flat"]}


def run(st):
    if own:
        return _own(st)
    if st["op"] == "heads":
        return _plain_heads(st) if st["way"] == "fwd" else _plain_heads_bwd(st)
    if st["op"] == "resnorm":
        return _plain_resnorm(st) if st["way"] == "fwd" else _plain_resnorm_bwd(st)
    return _plain_clip(st)


# -------------------------------------------------------------------- work
def work(case):
    size = {"bf16": 2, "fp32": 4}
    if case["op"] == "heads":
        n = case["B"] * case["N"] * case["H"] * case["d"]
        s = size[case["dtype"]]
        if case["way"] == "fwd":
            return {"bytes": 3 * n * (s + 2), "flops": 12 * n}
        read = 2 if case["norm"] != "none" else 0
        return {"bytes": 3 * n * (s + 2) + read * n * s, "flops": 24 * n}
    if case["op"] == "resnorm":
        n = case["B"] * case["N"] * case["C"]
        mods = 4 * case["C"] * ((1 if case["affine"] else 3) * case["B"] * case["frames"]
                                + (2 if case["affine"] else 0))
        sx, sb = size[case["x"]], size[case["branch"]]
        if case["way"] == "fwd":
            return {"bytes": 2 * n * (sx + sb) + mods, "flops": 10 * n}
        return {"bytes": 3 * n * (sx + sb) + 2 * mods, "flops": 24 * n}
    n = sum(math.prod(s) for s in _clip_shapes(case))
    return {"bytes": 2 * n * size[case["dtype"]], "flops": 3 * n}


# ------------------------------------------------------------------- exact
def _turn(st, b):
    """e^(i angle) of sample b's tokens: [N, 1, d / 2] complex."""
    N, d = st["N"], st["d"]
    p = torch.zeros(N, 3, dtype=torch.float64, device="cuda")
    if st["pos"] is not None:
        p = st["pos"][b].double()
    else:
        t, h, w = st["grid"][b].tolist()
        axes = [torch.arange(n, dtype=torch.float64, device="cuda") for n in (t, h, w)]
        p[:t * h * w] = torch.cartesian_prod(*axes).view(-1, 3)
    parts = []
    for a, n in enumerate(_pairs(d)):
        j = torch.arange(n, dtype=torch.float64, device="cuda")
        parts.append(p[:, a, None] * torch.exp(-j / n * math.log(THETA)))
    angle = torch.cat(parts, -1)[:, None]
    return torch.polar(torch.ones_like(angle), angle)


def _exact_heads(st, leaves):
    out = []
    for x, w in leaves:
        x = x.double() if not x.requires_grad else x
        if w is not None:
            dims = (2, 3) if st["norm"] == "token" else (3,)
            x = x / torch.sqrt(x.pow(2).mean(dims, keepdim=True) + EPS)
            x = x * (w.view(st["H"], st["d"]) if st["norm"] == "token" else w)
        rows = []
        for b in range(st["B"]):
            if st["interleaved"]:
                z = torch.view_as_complex(x[b].unflatten(-1, (-1, 2)).contiguous())
                rows.append(torch.view_as_real(z * _turn(st, b)).flatten(-2))
            else:
                half = st["d"] // 2
                z = torch.complex(x[b, ..., :half].contiguous(), x[b, ..., half:].contiguous())
                z = z * _turn(st, b)
                rows.append(torch.cat([z.real, z.imag], -1))
        out.append(torch.stack(rows).permute(0, 2, 1, 3))
    return out


def _exact_resnorm(st, x, b, gate, scale, shift, post):
    B, N, C, F = (st[k] for k in ("B", "N", "C", "frames"))

    def grouped(t):
        return t.reshape(B, F, N // F, C)

    def each(m):
        return m if m.dim() == 1 else m[:, :, None]

    b = grouped(b)
    if post is not None:
        b = post * b / torch.sqrt((b * b).mean(-1, keepdim=True) + EPS)
    y = grouped(x) + each(gate) * b
    if st["norm"] == "layer":
        var, mean = torch.var_mean(y, -1, correction=0, keepdim=True)
        z = (y - mean) / torch.sqrt(var + EPS)
    else:
        z = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS)
    h = z * ((0 if st["affine"] else 1) + each(scale)) + each(shift)
    return y.reshape(B, N, C), h.reshape(B, N, C)


def exact(case, seed):
    st = prepare(case, seed)
    f64 = lambda t: None if t is None else t.double()  # noqa: E731
    leaf = lambda t: None if t is None else t.double().requires_grad_(True)  # noqa: E731
    if case["op"] == "heads":
        if case["way"] == "fwd":
            q, k = _exact_heads(st, [(f64(st["q"]), f64(st["wq"])), (f64(st["k"]), f64(st["wk"]))])
            return {"q": q, "k": k, "v": st["v"].double().permute(0, 2, 1, 3)}
        q, k, wq, wk = leaf(st["q"]), leaf(st["k"]), leaf(st["wq"]), leaf(st["wk"])
        torch.autograd.backward(_exact_heads(st, [(q, wq), (k, wk)]), [f64(st["dq"]), f64(st["dk"])])
        parts = [q.grad, k.grad, st["dv"].double().permute(0, 2, 1, 3)]
        return {"dqkv": torch.cat([p.flatten(2) for p in parts], -1),
                "dw": [w.grad for w in (wq, wk) if w is not None]}
    if case["op"] == "resnorm":
        names = ("x", "b", "gate", "scale", "shift", "post")
        if case["way"] == "fwd":
            y, h = _exact_resnorm(st, *(f64(st[n]) for n in names))
            return {"y": y, "h": h}
        ins = [leaf(st[n]) for n in names]
        torch.autograd.backward(_exact_resnorm(st, *ins), [f64(st["dy"]), f64(st["dh"])])
        return {"d" + n: t.grad for n, t in zip(names, ins) if t is not None}
    total = math.fsum(float(torch.dot(g.double().flatten(), g.double().flatten()))
                      for g in st["grads"])
    norm = math.sqrt(total)
    flat = torch.zeros(st["places"][-1], dtype=torch.float64, device="cuda")
    for g, p in zip(st["grads"], st["places"]):
        flat[p:p + g.numel()] = g.double().flatten() * min(1.0, case["max_norm"] / (norm + EPS))
    return {"norm": torch.tensor(norm, dtype=torch.float64), "grads": flat}
