"""Cases of what a fine-tuning step of a video transformer does beside its sparse attention.

* ``cross``: attention of video tokens over a context (text and image tokens): queries
  [B, H, N, d], keys and values [Bk, Hk, M, d] with Hk dividing H and Bk 1 (one context for the
  whole batch) or B, and the first ``len`` context tokens of each sample valid (a sample without
  any gets zeros); its output and log-sum-exp, and its gradients with the probabilities computed
  again from them.
* ``ortho``: matrices to (nearly) orthogonal ones: X = G / (|G| + eps), then ``steps`` times
  X <- a X + (b A + c A A) X with A = X X^T (the transposed form for tall matrices).
* ``muon``: an optimiser step on matrices: m <- mu m + g, the orthogonalised g + mu m, and
  w <- (1 - lr decay) w - lr sqrt(max(1, rows / columns)) times it.

``own = False`` computes them in elementary torch operations in 32 bits, rounded once at the end;
``own = True`` calls the library.
"""

import math

import torch

own = False

EPS = 1e-7
COEFF = (3.4445, -4.7750, 2.0315)
STEPS, MU, LR, DECAY = 5, 0.95, 0.02, 0.01
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases
def _cross(name, way, B, Bk, H, Hk, N, M, d, lens="full", layout="heads"):
    """``lens`` "ragged": the samples' contexts get shorter one by one, "empty": the last has none.
    ``layout`` "tokens": every tensor lies as the projections leave it, [B, tokens, heads, d]."""
    return {"name": name, "op": "cross", "way": way, "B": B, "Bk": Bk, "H": H, "Hk": Hk, "N": N,
            "M": M, "d": d, "lens": lens, "layout": layout}


def _matrices(name, op, shapes, layers, dtype):
    """``layers`` times the matrices of ``shapes`` ("256x128 256x512 ...")."""
    return {"name": name, "op": op, "shapes": shapes, "layers": layers, "dtype": dtype}


BLOCK = "1536x1536 1536x1536 1536x1536 1536x1536 6144x1536 1536x6144"


def listed():
    return [
        # a test block's tokens over a short prompt: latency
        _cross("cross_small_fwd", "fwd", 1, 1, 2, 2, 100, 33, 64, "full", "tokens"),
        # the 480p video shape over a padded prompt of 512 tokens
        _cross("cross_480p_fwd", "fwd", 1, 1, 12, 12, 32760, 512, 128, "full", "tokens"),
        _cross("cross_480p_bwd", "bwd", 1, 1, 12, 12, 32760, 512, 128, "full", "tokens"),
        # the 720p video shape
        _cross("cross_720p_fwd", "fwd", 1, 1, 40, 40, 75600, 512, 128),
        # a batch of clips over prompts of different lengths, one dropped for guidance; grouped heads
        _cross("cross_ragged_bwd", "bwd", 3, 3, 8, 2, 5001, 257, 64, "empty", "tokens"),
        # four noise samples over one prompt and the tokens of one image
        _cross("cross_shared_bwd", "bwd", 4, 1, 12, 12, 3900, 769, 128),
        # one query token that pools a video's tokens (the head of a critic)
        _cross("cross_pool_fwd", "fwd", 2, 2, 12, 12, 1, 32760, 128, "ragged", "tokens"),
        # the four projections of a test block: latency
        _matrices("muon_small", "muon", "128x128 128x128 128x128 128x128", 1, "fp32"),
        # the attention projections of one 480p block, fp32 weights
        _matrices("muon_480p", "muon", "1536x1536 1536x1536 1536x1536 1536x1536", 1, "fp32"),
        # odd shapes: low-rank adapters, a patch embedding, a narrow head
        _matrices("ortho_odd", "ortho", "1536x24 16x5120 700x333 64x1001 1x77 129x129", 1, "fp32"),
        # one block with its MLP, and a stack of blocks
        _matrices("ortho_block", "ortho", BLOCK, 1, "bf16"),
        _matrices("ortho_stack", "ortho", BLOCK, 8, "bf16"),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    case = _draw(rng)
    del case["name"]
    return case


def _draw(rng):
    if rng.random() < 0.6:
        d = rng.choice([64, 128])
        H = rng.randint(1, 24)
        Hk = H // rng.choice([f for f in (1, 1, 1, 2, 3, 4) if H % f == 0])
        B = rng.choice([1, 1, 2, 3, 4])
        Bk = rng.choice([1, B])
        way = rng.choice(["fwd", "bwd"])
        # products of one pass, and values of its tensors, below those of the largest listed case
        most = (700_000_000 if way == "fwd" else 280_000_000) // (B * H)
        if rng.random() < 0.2:  # few queries over many keys
            N = _spread(rng, 1, 128)
            M = _spread(rng, 1000, min(32760, most // N, 100_000_000 // (Bk * Hk * d)))
        else:
            # (the logits of a single key have no gradient: only rounding is left of it)
            M = _spread(rng, 1 if way == "fwd" else 2, 1500)
            N = _spread(rng, 1, max(1, min(32760, most // M, 100_000_000 // (B * H * d))))
        return _cross("", way, B, Bk, H, Hk, N, M, d, rng.choice(["full", "ragged", "empty"]),
                      rng.choice(["heads", "tokens"]))
    count = rng.choice([1, 2, 5])
    dtype = rng.choice(["bf16", "fp32"])
    wide = 2048 if dtype == "fp32" else 6144
    shapes = []
    for _ in range(count):
        r = _spread(rng, 1, 2048)
        c = rng.choice([r, _spread(rng, 1, wide)])
        shapes.append("%dx%d" % rng.choice([(r, c), (c, r)]))
    return _matrices("", rng.choice(["ortho", "muon"]), " ".join(shapes), rng.choice([1, 1, 2]),
                     dtype)


def _lens(case):
    """Valid context tokens of each sample; None: all of them."""
    B, M = case["B"], case["M"]
    if case["lens"] == "full":
        return None
    lens = [max(1, M - (M // (B + 1)) * b - b) for b in range(B)]
    if case["lens"] == "empty" and B > 1:
        lens[-1] = 0
    return lens


def _shapes(case):
    return [tuple(int(n) for n in s.split("x")) for s in case["shapes"].split()] * case["layers"]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape, dtype=torch.float32, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda").mul_(std).to(dtype)

    st = dict(case)
    if case["op"] == "cross":
        B, Bk, H, Hk, N, M, d = (case[k] for k in ("B", "Bk", "H", "Hk", "N", "M", "d"))
        tokens = case["layout"] == "tokens"

        def heads(b, h, n):
            if tokens:
                return rand(b, n, h, d, dtype=torch.bfloat16).transpose(1, 2)
            return rand(b, h, n, d, dtype=torch.bfloat16)

        st["q"], st["k"], st["v"] = heads(B, H, N), heads(Bk, Hk, M), heads(Bk, Hk, M)
        # the first context token draws every query a little
        pull = rand(H, d, std=0.2)
        st["q"] += pull[:, None].to(torch.bfloat16)
        st["k"][:, :, :1] += (20 / d ** 0.5 * pull[::H // Hk, None]).to(torch.bfloat16)
        lens = _lens(case)
        st["len"] = torch.tensor(lens, dtype=torch.int32, device="cuda") if lens else None
        if case["way"] == "bwd":
            st["do"] = heads(B, H, N)
            o, st["lse"] = _attention(st)  # what the forward left
            st["o"] = _laid(o, tokens)
        return st
    dtype = TYPES[case["dtype"]]
    st["g"] = []
    for r, c in _shapes(case):
        # a gradient: a few strong directions and noise
        k = min(8, r, c)
        g = rand(r, k) @ (rand(k, c) * torch.logspace(0, -1, k, device="cuda")[:, None])
        st["g"].append((g.mul_(0.3).add_(rand(r, c)).mul_(1e-3)).to(dtype))
    if case["op"] == "muon":
        st["m"] = [rand(*g.shape, std=1e-2) for g in st["g"]]
        st["w"] = [rand(*g.shape, std=g.shape[1] ** -0.5).to(dtype) for g in st["g"]]
    return st


def _laid(t, tokens):
    """[B, H, n, d] in bf16, as values or as the view of [B, n, H, d]."""
    if tokens:
        return t.transpose(1, 2).to(torch.bfloat16).contiguous().transpose(1, 2)
    return t.to(torch.bfloat16)


# ---------------------------------------------------------------- plain form
def _probabilities(st):
    """(P, log-sum-exp, q, k, v) in 32 bits, heads grouped: [B, Hk, H / Hk, ...]."""
    Hk, M, d = st["Hk"], st["M"], st["d"]
    q = st["q"].float().unflatten(1, (Hk, -1))
    k, v = st["k"].float()[:, :, None], st["v"].float()[:, :, None]
    s = (q @ k.transpose(-1, -2)).mul_(d ** -0.5)
    if st["len"] is not None:
        behind = torch.arange(M, device="cuda") >= st["len"][:, None]
        s.masked_fill_(behind[:, None, None, None], -math.inf)
    top = s.amax(-1, keepdim=True).clamp_min_(-1e30)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (total.log() + top).squeeze(-1).flatten(1, 2)
    p.div_(total.masked_fill(total == 0, 1.0))
    return p, lse, q, k, v


def _attention(st):
    p, lse, _, _, v = _probabilities(st)
    return (p @ v).flatten(1, 2), lse


def _plain_cross(st):
    tokens = st["layout"] == "tokens"
    if st["way"] == "fwd":
        o, lse = _attention(st)
        return {"o": _laid(o, tokens), "lse": lse}
    p, _, q, k, v = _probabilities(st)
    do = st["do"].float().unflatten(1, (st["Hk"], -1))
    shared = (0, 2) if st["Bk"] < st["B"] else (2,)
    dv = (p.transpose(-1, -2) @ do).sum(shared, keepdim=True)
    ds = do @ v.transpose(-1, -2)
    ds.sub_((ds * p).sum(-1, keepdim=True)).mul_(p).mul_(st["d"] ** -0.5)
    dq = (ds @ k).flatten(1, 2)
    dk = (ds.transpose(-1, -2) @ q).sum(shared, keepdim=True)
    return {"dq": _laid(dq, tokens), "dk": _laid(dk[:, :, 0], tokens),
            "dv": _laid(dv[:, :, 0], tokens)}


def _plain_ortho(g):
    a, b, c = COEFF
    x = g.float()
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.t()
    x = x / (x.norm() + EPS)
    for _ in range(STEPS):
        A = x @ x.t()
        x = a * x + (b * A + c * (A @ A)) @ x
    return x.t() if tall else x


def _plain_muon(st):
    for w, g, m in zip(st["w"], st["g"], st["m"]):
        m.mul_(MU).add_(g.float())
        o = _plain_ortho(g.float() + MU * m)
        step = LR * math.sqrt(max(1.0, w.shape[0] / w.shape[1]))
        w.copy_((1 - LR * DECAY) * w.float() - step * o)
    return {"w": st["w"], "m": st["m"]}


# --------------------------------------------------------------- the library
def _own(st):
    import block_sparse_attention_sparge_gb300 as S
    if st["op"] == "ortho":
        return S.sparge_orthogonalize(st["g"], steps=STEPS, coefficients=COEFF, eps=EPS)
    if st["op"] == "muon":
        S.sparge_muon_step(st["w"], st["g"], st["m"], lr=LR, momentum=MU, weight_decay=DECAY,
                           steps=STEPS, coefficients=COEFF, eps=EPS)
        return {"w": st["w"], "m": st["m"]}
    q, k, v = st["q"], st["k"], st["v"]
    if st["way"] == "fwd":
        # (the results lie as the inputs do)
        o, lse = S.sparge_cross_fwd(q, k, v, st["len"], out=torch.empty_like(q))
        return {"o": o, "lse": lse}
    dq, dk, dv = S.sparge_cross_bwd(q, k, v, st["o"], st["lse"], st["do"], st["len"],
                                    out=(torch.empty_like(q), torch.empty_like(k),
                                         torch.empty_like(v)))
    return {"dq": dq, "dk": dk, "dv": dv}


def run(st):
    if own:
        return _own(st)
    if st["op"] == "cross":
        return _plain_cross(st)
    if st["op"] == "ortho":
        return [_plain_ortho(g).to(g.dtype) for g in st["g"]]
    return _plain_muon(st)


# -------------------------------------------------------------------- work
def work(case):
    if case["op"] == "cross":
        B, Bk, H, Hk, N, M, d = (case[k] for k in ("B", "Bk", "H", "Hk", "N", "M", "d"))
        lens = _lens(case) or [M] * B
        q = 2 * B * H * N * d
        kv = 2 * Hk * d * (sum(lens) if Bk == B else max(lens))
        whole = 2 * Bk * Hk * M * d  # gradients are written for every context token
        pairs = H * N * sum(lens)
        if case["way"] == "fwd":
            return {"bytes": 2 * q + 2 * kv + 4 * B * H * N, "flops": 4 * pairs * d}
        return {"bytes": 4 * q + 2 * kv + 2 * whole + 4 * B * H * N, "flops": 10 * pairs * d}
    size = {"bf16": 2, "fp32": 4}[case["dtype"]]
    byte = flops = 0
    for r, c in _shapes(case):
        m, n = min(r, c), max(r, c)
        byte += r * c * (2 * size if case["op"] == "ortho" else 3 * size + 8)
        # A and A A are symmetric: half of them; then (...) X
        flops += STEPS * (m * m * n + m * m * m + 2 * m * m * n)
    return {"bytes": byte, "flops": flops}


# ------------------------------------------------------------------- exact
def _exact_head(q, k, v, n, do):
    """One head of one sample in 64 bits: output, log-sum-exp and, with ``do``, the gradients
    (zeros behind the n valid tokens)."""
    if n == 0:
        zeros = [torch.zeros_like(t) for t in (q, q, k, v)]
        return zeros[0], q.new_full((q.shape[0],), -math.inf), *zeros[1:]
    q, kn, vn = (t.detach().requires_grad_(do is not None) for t in (q, k[:n], v[:n]))
    logits = torch.einsum("id,jd->ij", q, kn) / math.sqrt(q.shape[1])
    lse = torch.logsumexp(logits, 1)
    o = torch.einsum("ij,jd->id", torch.exp(logits - lse[:, None]), vn)
    if do is None:
        return o, lse, None, None, None
    dq, dk, dv = torch.autograd.grad(o, (q, kn, vn), do)
    pad = (0, 0, 0, k.shape[0] - n)
    return (o.detach(), lse.detach(), dq, torch.nn.functional.pad(dk, pad),
            torch.nn.functional.pad(dv, pad))


def _exact_cross(st):
    B, Bk, H, Hk = (st[k] for k in ("B", "Bk", "H", "Hk"))
    bwd = st["way"] == "bwd"
    q64 = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = q64[..., 0].clone()
    dk = torch.zeros(st["k"].shape, dtype=torch.float64, device="cuda")
    dv = torch.zeros_like(dk)
    lens = _lens(st) or [st["M"]] * B
    for b in range(B):
        for h in range(H):
            at = (b if Bk > 1 else 0, h // (H // Hk))
            got = _exact_head(st["q"][b, h].double(), st["k"][at].double(), st["v"][at].double(),
                              lens[b], st["do"][b, h].double() if bwd else None)
            lse[b, h] = got[1]
            if bwd:
                q64[b, h] = got[2]
                dk[at] += got[3]
                dv[at] += got[4]
            else:
                q64[b, h] = got[0]
    return {"dq": q64, "dk": dk, "dv": dv} if bwd else {"o": q64, "lse": lse}


def _exact_ortho(g):
    """By the Gram matrix of the short side: the iteration multiplies X by polynomials of it."""
    a, b, c = COEFF
    x = g.double()
    short = 0 if x.shape[0] <= x.shape[1] else 1
    x = x / (torch.linalg.norm(x) + EPS)
    eye = torch.eye(x.shape[short], dtype=torch.float64, device=x.device)
    gram = x.mm(x.mT) if short == 0 else x.mT.mm(x)
    whole = eye
    for _ in range(STEPS):
        f = a * eye + gram.mm(b * eye + c * gram)  # commutes with the Gram matrix
        whole = f.mm(whole)
        gram = f.mm(gram).mm(f)
    return whole.mm(x) if short == 0 else x.mm(whole)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "cross":
        return _exact_cross(st)
    if case["op"] == "ortho":
        return [_exact_ortho(g) for g in st["g"]]
    out = {"w": [], "m": []}
    for w, g, m in zip(st["w"], st["g"], st["m"]):
        m = MU * m.double() + g.double()
        o = _exact_ortho(g.double() + MU * m)
        gain = math.sqrt(max(1.0, w.shape[0] / w.shape[1]))
        out["w"].append(w.double() * (1 - LR * DECAY) - LR * gain * o)
        out["m"].append(m)
    return out
