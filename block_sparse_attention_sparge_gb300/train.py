"""Trainable block-sparse attention on the library's kernels, and one
velocity-distillation training step at the level of an attention block.

Method: the page "SpargeAttention2: Trainable Sparse Attention via Hybrid
Top-k+Top-p Masking and Distillation Fine-Tuning", section "Abstract" (the
sparse attention is trainable and fine-tuned with a distillation objective),
and the mindverse page "Optimierung der Effizienz von Video-Diffusionsmodellen
durch SpargeAttention2", sections "Velocity Distillation Loss" (a frozen model
with full attention is the teacher, the sparse model the student, and the
student is fitted to the teacher's outputs instead of to the data) and
"Effiziente Kernel-Implementierung und Modellanpassung" (every attention layer
is replaced by the sparse one, then fine-tuned with that loss).

No diffusion model, weights or data exist here, so this module holds the
mechanics only: ``SparseAttentionFunction`` is a torch.autograd.Function whose
forward and backward are ``sparge_attn_fwd`` / ``sparge_attn_bwd``; the mask is
built from Q and K by ``sparge_mask`` and held constant (the selection is
piecewise constant, so no gradient flows through it). ``AttentionBlock`` is a
multi-head attention block (Q/K/V and output projections) whose attention is
either that sparse function or the same kernels with every block kept (dense).
``distillation_step`` runs one optimiser step of a student block against a
frozen dense teacher on the same input, with the mean squared error of the two
outputs as the loss. Projections run in torch (cuBLAS); every attention step
runs in the library's kernels. There is no CPU path: the binding raises when
the library or a GPU is missing.

What surrounds the attention in a block of a video transformer is here too, as
autograd functions over the library: ``qkv_heads`` (RMS norm of Q and K, rotary
positions over time, height and width, and the attention's layout),
``residual_norm`` (gated residual join and the modulated norm that follows it)
and ``clip_grad_norm_``. ``AttentionBlock`` uses the first two when it is given
a rope or a norm, ``BlockStack`` joins each block's residual with the next
block's norm, and ``distillation_step`` clips when it is given a bound.
"""

from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import binding as B


def _gradient(g, dtype):
    """A gradient as the library reads it: dense, of the given type, on a 16-byte
    boundary. Autograd hands over views that begin anywhere (the pieces of a
    concatenation's gradient), which are contiguous already."""
    g = g.to(dtype).contiguous()
    return g if g.data_ptr() % 16 == 0 else g.clone()


class SparseAttentionFunction(torch.autograd.Function):
    """O = block-sparse attention(Q, K, V) under a fixed block mask.

    Inputs are bf16 [B, H, N, d] CUDA tensors; the mask is given as the CSR
    and CSC lists ``sparge_mask`` returns. Gradients flow to Q, K and V."""

    @staticmethod
    def forward(ctx, q, k, v, row_idx, row_cnt, col_idx, col_cnt, softmax_scale):
        q, k, v = (t.contiguous() for t in (q, k, v))
        o, lse = B.sparge_attn_fwd(q, k, v, row_idx, row_cnt, softmax_scale)
        ctx.save_for_backward(q, k, v, o, lse, row_idx, row_cnt, col_idx, col_cnt)
        ctx.softmax_scale = softmax_scale
        return o

    @staticmethod
    def backward(ctx, dout):
        q, k, v, o, lse, row_idx, row_cnt, col_idx, col_cnt = ctx.saved_tensors
        dout = _gradient(dout, torch.bfloat16)
        dq, dk, dv = B.sparge_attn_bwd(q, k, v, o, lse, dout, row_idx, row_cnt, col_idx,
                                       col_cnt, ctx.softmax_scale)
        return dq, dk, dv, None, None, None, None, None


def sparse_attention(q, k, v, k_frac: float, p: float, softmax_scale: float = 0.0):
    """Hybrid-masked attention with autograd: the mask (Top-k fraction
    ``k_frac``, Top-p ``p``) is computed from the current Q and K, then held
    constant for the forward and backward of this call. ``k_frac = 1`` keeps
    every block (dense attention)."""
    with torch.no_grad():
        m = B.sparge_mask(q.detach().contiguous(), k.detach().contiguous(), k_frac, p,
                          softmax_scale, want_csc=True)
    return SparseAttentionFunction.apply(q, k, v, m["row_idx"], m["row_cnt"], m["col_idx"],
                                         m["col_cnt"], softmax_scale)


class HeadsFunction(torch.autograd.Function):
    """``sparge_heads_fwd`` with the gradients of ``sparge_heads_bwd``."""

    @staticmethod
    def forward(ctx, q, k, v, q_weight, k_weight, grid, pos, rope, norm, eps):
        ctx.set_materialize_grads(False)
        keep = norm is not None
        ctx.save_for_backward(q if keep else None, k if keep else None, q_weight, k_weight, grid,
                              pos)
        ctx.how = dict(rope=rope, norm=norm, eps=eps)
        ctx.dtype = next((t.dtype for t in (q, k, v) if t is not None), None)
        return B.sparge_heads_fwd(q, k, v, rope=rope, grid=grid, pos=pos, norm=norm,
                                  q_weight=q_weight, k_weight=k_weight, eps=eps)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk, dv):
        q, k, wq, wk, grid, pos = ctx.saved_tensors
        need = ctx.needs_input_grad
        wanted = (need[0] or need[3], need[1] or need[4], need[2])
        dq, dk, dv = (_gradient(g, torch.bfloat16) if g is not None and w else None
                      for g, w in zip((dq, dk, dv), wanted))
        if dq is None and dk is None and dv is None:
            return (None,) * 10
        grads = B.sparge_heads_bwd(dq, dk, dv, q if dq is not None else None,
                                   k if dk is not None else None, grid=grid, pos=pos,
                                   q_weight=wq if dq is not None else None,
                                   k_weight=wk if dk is not None else None, dtype=ctx.dtype,
                                   **ctx.how)
        return (*(g if w else None for g, w in zip(grads, need)), *(None,) * 5)


def qkv_heads(q=None, k=None, v=None, rope: B.RopeAxes | None = None, grid=None, pos=None,
              norm: str | None = None, q_weight=None, k_weight=None, eps: float = 1e-6):
    """Projections [B, N, H, d] to the attention's bf16 [B, H, N, d], with
    autograd: see ``sparge_heads_fwd``. Gradients flow to q, k, v and the norm
    weights."""
    return HeadsFunction.apply(q, k, v, q_weight, k_weight, grid, pos, rope, norm, eps)


class ResidualNormFunction(torch.autograd.Function):
    """``sparge_resnorm_fwd`` with the gradients of ``sparge_resnorm_bwd``;
    returns (y, h), None for y without a branch and for h without a norm."""

    @staticmethod
    def forward(ctx, x, branch, gate, scale, shift, post_weight, norm, unit_offset, eps, h_dtype):
        ctx.set_materialize_grads(False)
        y, h, stats = B.sparge_resnorm_fwd(x, branch, gate, scale, shift, norm, unit_offset,
                                           post_weight, eps, h_dtype)
        ctx.save_for_backward(x, branch, gate, scale, shift, post_weight, stats)
        ctx.how = dict(norm=norm, unit_offset=unit_offset)
        ctx.h_dtype = h.dtype if h is not None else None
        return (y if branch is not None else None), h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        x, branch, gate, scale, shift, post_weight, stats = ctx.saved_tensors
        need = ctx.needs_input_grad
        if dy is None and dh is None:
            return (None,) * 10
        dy = _gradient(dy, x.dtype) if dy is not None else None
        dh = _gradient(dh, ctx.h_dtype) if dh is not None else None
        grads = B.sparge_resnorm_bwd(dy, dh, x, branch, gate, scale, shift, stats,
                                     post_weight=post_weight, want_mods=any(need[2:6]), **ctx.how)
        return (*(g if w else None for g, w in zip(grads, need)), *(None,) * 4)


def residual_norm(x, branch=None, gate=None, scale=None, shift=None, norm: str | None = "layer",
                  unit_offset: bool = True, post_weight=None, eps: float = 1e-6, h_dtype=None):
    """(y, h) = (x + gate * branch, norm(y) * (1 + scale) + shift), with
    autograd: see ``sparge_resnorm_fwd``. y is x itself without a branch, h is
    None without a norm."""
    y, h = ResidualNormFunction.apply(x, branch, gate, scale, shift, post_weight, norm,
                                      unit_offset, eps, h_dtype)
    return (x if branch is None else y), h


def clip_grad_norm_(parameters, max_norm: float, eps: float = 1e-6) -> torch.Tensor:
    """Scales the parameters' gradients in place so that their global 2-norm is
    at most ``max_norm``; returns the norm before (an fp32 scalar tensor on the
    device: nothing waits for the GPU)."""
    if isinstance(parameters, torch.Tensor):
        parameters = [parameters]
    grads = [p.grad for p in parameters if p.grad is not None]
    if not grads:
        return torch.zeros(())
    return B.sparge_clip_grads(grads, max_norm, eps=eps)


class AttentionBlock(torch.nn.Module):
    """Multi-head attention block on tokens x [B, N, C]: Q, K, V projections
    to H heads of width d, attention, output projection back to C. Weights are
    fp32; the attention runs in bf16 through the library.

    ``k_frac`` and ``p`` select the hybrid mask; ``k_frac = 1`` gives dense
    attention (every block kept). ``rope`` turns Q and K by the tokens'
    positions on the ``grid`` given to ``forward`` (int32 [B, 3]); ``qk_norm``
    ("token" or "head") is their RMS norm, with learned weights. With ``norm``
    ("layer" or "rms") the block is residual: x + gate * attention(norm(x) * (1
    + scale) + shift), where ``modulation`` [B, F, 3, C] (fp32) holds shift,
    scale and gate for each run of N / F tokens, or is absent."""

    def __init__(self, channels: int, heads: int, head_dim: int, k_frac: float = 1.0,
                 p: float = 0.0, generator: torch.Generator | None = None, device="cuda",
                 rope: B.RopeAxes | None = None, qk_norm: str | None = None,
                 norm: str | None = None):
        super().__init__()
        self.rope, self.qk_norm, self.norm = rope, qk_norm, norm
        self.heads, self.head_dim = heads, head_dim
        self.k_frac, self.p = k_frac, p
        inner = heads * head_dim
        std = channels ** -0.5

        def weight(rows, cols):
            w = torch.randn((rows, cols), generator=generator) * std
            return torch.nn.Parameter(w.to(device))

        self.wq = weight(channels, inner)
        self.wk = weight(channels, inner)
        self.wv = weight(channels, inner)
        self.wo = torch.nn.Parameter((torch.randn((inner, channels), generator=generator)
                                      * inner ** -0.5).to(device))
        if qk_norm is not None:
            width = inner if qk_norm == "token" else head_dim
            self.norm_q, self.norm_k = (torch.nn.Parameter(torch.ones(width, device=device))
                                        for _ in range(2))

    def _heads(self, t, b, n):
        return (t.reshape(b, n, self.heads, self.head_dim).permute(0, 2, 1, 3)
                .to(torch.bfloat16).contiguous())

    def attend(self, x, grid=None):
        """The attention of tokens x, without the residual and its norm."""
        b, n, _ = x.shape
        if self.rope is None and self.qk_norm is None:
            q = self._heads(x @ self.wq, b, n)
            k = self._heads(x @ self.wk, b, n)
            v = self._heads(x @ self.wv, b, n)
        else:
            split = (b, n, self.heads, self.head_dim)
            normed = self.qk_norm is not None
            q, k, v = qkv_heads((x @ self.wq).view(split), (x @ self.wk).view(split),
                                (x @ self.wv).view(split), self.rope,
                                grid if self.rope is not None else None, None, self.qk_norm,
                                self.norm_q if normed else None, self.norm_k if normed else None)
        o = sparse_attention(q, k, v, self.k_frac, self.p)
        o = o.float().permute(0, 2, 1, 3).reshape(b, n, self.heads * self.head_dim)
        return o @ self.wo

    def forward(self, x, grid=None, modulation=None):
        if self.norm is None:
            if modulation is not None:
                raise ValueError("a modulation needs a block with a norm")
            return self.attend(x, grid)
        return run_blocks([self], x, grid,
                          modulation[:, :, None] if modulation is not None else None)


def run_blocks(blocks, x, grid=None, modulation=None):
    """Residual blocks one after another, each block's join in one pass with the
    next block's norm. ``modulation`` is fp32 [B, F, blocks, 3, C]: shift, scale
    and gate of each block, or None."""
    def mod(i, k):
        return modulation[:, :, i, k] if modulation is not None else None

    _, h = residual_norm(x, None, None, mod(0, 1), mod(0, 0), blocks[0].norm)
    for i, block in enumerate(blocks):
        o = block.attend(h, grid)
        if i + 1 < len(blocks):
            x, h = residual_norm(x, o, mod(i, 2), mod(i + 1, 1), mod(i + 1, 0),
                                 blocks[i + 1].norm)
        else:
            x, _ = residual_norm(x, o, mod(i, 2), norm=None)
    return x


class BlockStack(torch.nn.Module):
    """Residual attention blocks in a row (``run_blocks``)."""

    def __init__(self, blocks):
        super().__init__()
        self.blocks = torch.nn.ModuleList(blocks)
        if len(self.blocks) == 0 or any(b.norm is None for b in self.blocks):
            raise ValueError("expected blocks with a norm")

    def forward(self, x, grid=None, modulation=None):
        return run_blocks(self.blocks, x, grid, modulation)


def distillation_step(student, teacher, x: torch.Tensor, optimizer: torch.optim.Optimizer,
                      max_grad_norm: float | None = None, **inputs) -> float:
    """One fine-tuning step of the sparse student against the frozen dense
    teacher: loss = mean((student(x) - teacher(x))^2); backward through the
    library's sparse attention backward; gradients clipped to the global norm
    ``max_grad_norm`` where that is given; optimiser step. ``inputs`` (grid,
    modulation) go to both. Returns the loss."""
    with torch.no_grad():
        target = teacher(x, **inputs)
    optimizer.zero_grad(set_to_none=True)
    loss = torch.mean((student(x, **inputs) - target) ** 2)
    loss.backward()
    if max_grad_norm is not None:
        clip_grad_norm_(student.parameters(), max_grad_norm)
    optimizer.step()
    return float(loss.item())
