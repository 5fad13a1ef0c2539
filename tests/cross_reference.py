"""Attention over a context in 64 bits, with bounds of what the kernels may be off.

The kernels multiply bf16 values and add in fp32.  They round P (and dS) to bf16 before the
second product, read O as it was rounded for D, and round each result once; a rounding is off
by at most HALF of the value.  Everything else (exponents, sums, the log-sum-exp) is fp32: its
part, for logits of a few tens over at most 128 channels, is below 2^-10 of the terms' sizes:
128 * 2^-23 of the sum of |q k| scale, at most some 20, is 2^-11.7 of a probability, twice
where the log-sum-exp has an error of its own.
"""

import torch

HALF = 2.0 ** -8   # of bf16
FP32 = 2.0 ** -10  # see above


def reference(q, k, v, lens=None, scale=None, dout=None):
    """o, lse and, with dout, dq, dk, dv, in 64 bits, and the bounds of o, dq, dk, dv."""
    B, H, N, d = q.shape
    Bk, Hk, M, _ = k.shape
    scale = d ** -0.5 if scale is None else scale
    out = {"o": q.new_zeros(q.shape, dtype=torch.float64),
           "lse": q.new_full((B, H, N), -float("inf"), dtype=torch.float64)}
    lim = {"o": torch.zeros_like(out["o"])}
    if dout is not None:
        for n, t in (("dq", q), ("dk", k), ("dv", v)):
            out[n] = torch.zeros(t.shape, dtype=torch.float64, device=q.device)
            lim[n] = torch.zeros_like(out[n])
    for b in range(B):
        n = M if lens is None else min(max(int(lens[b]), 0), M)
        if n == 0:
            continue
        for h in range(H):
            at = (b if Bk > 1 else 0, h // (H // Hk))
            Q, K, V = q[b, h].double(), k[at][:n].double(), v[at][:n].double()
            s = scale * (Q @ K.T)
            lse = s.logsumexp(-1)
            P = (s - lse[:, None]).exp()
            o = P @ V
            out["o"][b, h], out["lse"][b, h] = o, lse
            size = P @ V.abs()
            lim_o = HALF * (size + o.abs()) + FP32 * size
            lim["o"][b, h] = lim_o
            if dout is None:
                continue
            G = dout[b, h].double()
            dS = P * (G @ V.T - (G * o).sum(-1, keepdim=True))
            off_D = (G.abs() * lim_o).sum(-1, keepdim=True)
            terms = P * (G.abs() @ V.abs().T + (G * o).abs().sum(-1, keepdim=True))
            off = HALF * dS.abs() + P * off_D + FP32 * terms
            out["dq"][b, h] = scale * (dS @ K)
            lim["dq"][b, h] = abs(scale) * (off @ K.abs())
            out["dk"][at][:n] += scale * (dS.T @ Q)
            lim["dk"][at][:n] += abs(scale) * (off.T @ Q.abs())
            out["dv"][at][:n] += P.T @ G
            lim["dv"][at][:n] += (HALF + FP32) * (P.T @ G.abs())
    for n in ("dq", "dk", "dv"):
        if n in lim:
            lim[n] += HALF * out[n].abs()
    return out, lim


def check(got, out, lim, names):
    """Every element within its bound, and the whole within three roundings (P or dS, O, the
    result) in the 2-norm, which the bounds' worst cases do not show for long sums."""
    for n, t in zip(names, got):
        if n == "lse":
            fine = out[n].isfinite()
            assert torch.equal(t[~fine].double(), out[n][~fine])
            assert ((t[fine].double() - out[n][fine]).abs() <= FP32).all()
            continue
        assert t.dtype == torch.bfloat16 and t.shape == out[n].shape
        e = (t.double() - out[n]).abs()
        # 2^-133: the smallest step of bf16
        bad = ~(e <= lim[n] + 2.0 ** -133)
        assert not bad.any(), (n, int(bad.sum()), float((e / (lim[n] + 1e-30)).max()))
        norm = out[n].norm()
        # (a gradient that is a difference of equal terms has only its bound)
        if norm > 1e-3 * lim[n].norm() * 2 ** 8:
            assert e.norm() <= 3 * HALF * norm, (n, float(e.norm() / norm))
