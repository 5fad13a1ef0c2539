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

Between the self-attention and the next block stands the attention over a text or
image context: ``cross_attention`` with autograd, ``CrossAttentionBlock`` around it,
which ``BlockStack`` takes like any other block. ``Muon`` is an optimiser for the
blocks' matrices whose whole step runs in the library.
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


def _strided(t):
    """[batch, heads, tokens, d] in bf16 as the library reads it: any strides of
    multiples of 16 bytes, so views of projections [batch, tokens, heads, d] stay
    where they are; copied else (an expanded gradient, a view at an odd place)."""
    t = t.to(torch.bfloat16)
    *outer, last = t.stride()
    fits = (last == 1 and t.data_ptr() % 16 == 0
            and all(s > 0 and s % 8 == 0 for s, n in zip(outer, t.shape) if n > 1))
    return t if fits else t.clone(memory_format=torch.contiguous_format)


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


class CrossAttentionFunction(torch.autograd.Function):
    """``sparge_cross_fwd`` with the gradients of ``sparge_cross_bwd``; the output
    and the gradients lie as their inputs do."""

    @staticmethod
    def forward(ctx, q, k, v, kv_len, softmax_scale):
        ctx.dtypes = [t.dtype for t in (q, k, v)]
        q, k, v = (_strided(t) for t in (q, k, v))
        o, lse = B.sparge_cross_fwd(q, k, v, kv_len, softmax_scale, out=torch.empty_like(q))
        ctx.save_for_backward(q, k, v, o, lse, kv_len)
        ctx.softmax_scale = softmax_scale
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, k, v, o, lse, kv_len = ctx.saved_tensors
        grads = B.sparge_cross_bwd(q, k, v, o, lse, _strided(dout), kv_len, ctx.softmax_scale,
                                   out=[torch.empty_like(t) for t in (q, k, v)])
        return (*(g.to(t) for g, t in zip(grads, ctx.dtypes)), None, None)


def cross_attention(q, k, v, kv_len=None, softmax_scale: float = 0.0):
    """Attention of q [B, H, N, d] over the context k, v [Bk, Hk, M, d], with
    autograd: see ``sparge_cross_fwd``. Gradients flow to q, k and v."""
    return CrossAttentionFunction.apply(q, k, v, kv_len, softmax_scale)


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

    crosses = False  # whether run_blocks' context goes to it, and no row of its modulation

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


class CrossAttentionBlock(torch.nn.Module):
    """Attention of tokens x [B, N, C] over a context [B or 1, M, context_channels]:
    H query heads, ``kv_heads`` key heads (a divisor of H), projections in fp32, the
    attention in bf16 through the library. ``qk_norm`` ("token" or "head") is the RMS
    norm of Q and K, with learned weights. With ``norm`` ("layer" or "rms") the block
    is residual: x + attention(norm(x)). ``kv_len`` (int32 [B]) counts the valid
    context tokens of each sample."""

    crosses = True

    def __init__(self, channels: int, heads: int, head_dim: int, context_channels: int,
                 kv_heads: int | None = None, generator: torch.Generator | None = None,
                 device="cuda", qk_norm: str | None = None, norm: str | None = None):
        super().__init__()
        self.heads, self.head_dim, self.kv_heads = heads, head_dim, kv_heads or heads
        self.qk_norm, self.norm = qk_norm, norm
        inner, key_inner = heads * head_dim, self.kv_heads * head_dim

        def weight(rows, cols):
            w = torch.randn((rows, cols), generator=generator) * rows ** -0.5
            return torch.nn.Parameter(w.to(device))

        self.wq = weight(channels, inner)
        self.wk = weight(context_channels, key_inner)
        self.wv = weight(context_channels, key_inner)
        self.wo = weight(inner, channels)
        if qk_norm is not None:
            widths = (inner, key_inner) if qk_norm == "token" else (head_dim, head_dim)
            self.norm_q, self.norm_k = (torch.nn.Parameter(torch.ones(w, device=device))
                                        for w in widths)

    def _heads(self, t, heads):
        return t.unflatten(-1, (heads, self.head_dim))

    def attend(self, x, grid=None, context=None, kv_len=None):
        """The attention of tokens x, without the residual and its norm."""
        if context is None:
            raise ValueError("a cross attention block needs a context")
        q = self._heads(x @ self.wq, self.heads)
        k, v = (self._heads(context @ w, self.kv_heads) for w in (self.wk, self.wv))
        if self.qk_norm is None:
            q, k, v = (t.to(torch.bfloat16).transpose(1, 2) for t in (q, k, v))
        else:
            q, _, _ = qkv_heads(q, norm=self.qk_norm, q_weight=self.norm_q)
            _, k, v = qkv_heads(None, k, v, norm=self.qk_norm, k_weight=self.norm_k)
        o = cross_attention(q, k, v, kv_len)
        return o.transpose(1, 2).flatten(2).float() @ self.wo

    def forward(self, x, context, kv_len=None):
        if self.norm is None:
            return self.attend(x, None, context, kv_len)
        return run_blocks([self], x, context=context, kv_len=kv_len)


def run_blocks(blocks, x, grid=None, modulation=None, context=None, kv_len=None):
    """Residual blocks one after another, each block's join in one pass with the
    next block's norm. ``modulation`` is fp32 [B, F, blocks, 3, C]: shift, scale
    and gate of each block that takes one (attention over a context does not), or
    None. ``context`` and ``kv_len`` go to the blocks that attend to one."""
    crosses = [getattr(block, "crosses", False) for block in blocks]
    rows, count = [], 0
    for cross in crosses:
        rows.append(None if cross else count)
        count += not cross
    if modulation is not None and count < len(blocks) and modulation.shape[2] != count:
        raise ValueError(f"expected a modulation of {count} rows: {count} blocks take one, those "
                         "that attend to a context none")

    def mod(i, k):
        if modulation is None or rows[i] is None:
            return None
        return modulation[:, :, rows[i], k]

    _, h = residual_norm(x, None, None, mod(0, 1), mod(0, 0), blocks[0].norm)
    for i, block in enumerate(blocks):
        o = block.attend(h, grid, context, kv_len) if crosses[i] else block.attend(h, grid)
        if i + 1 < len(blocks):
            x, h = residual_norm(x, o, mod(i, 2), mod(i + 1, 1), mod(i + 1, 0),
                                 blocks[i + 1].norm)
        else:
            x, _ = residual_norm(x, o, mod(i, 2), norm=None)
    return x


class BlockStack(torch.nn.Module):
    """Residual blocks of self- and cross attention in a row (``run_blocks``)."""

    def __init__(self, blocks):
        super().__init__()
        self.blocks = torch.nn.ModuleList(blocks)
        if len(self.blocks) == 0 or any(b.norm is None for b in self.blocks):
            raise ValueError("expected blocks with a norm")

    def forward(self, x, grid=None, modulation=None, context=None, kv_len=None):
        return run_blocks(self.blocks, x, grid, modulation, context, kv_len)


class Muon(torch.optim.Optimizer):
    """Optimiser of matrices by orthogonalised momenta: ``sparge_muon_step`` over all
    parameters of a group at once. Momenta are fp32 whatever the parameters' type.
    ``half`` (the default here, where the binding goes by the parameters' type, as None
    does) takes the products in fp16: the update is off by some 2^-9 of its size, by more for
    narrow matrices with few strong directions (``include/sparge.h`` has the figures), whose
    groups may be given ``half=False``. A captured step keeps the learning rate and the other
    numbers of its capture.

    The gain sqrt(max(1, outputs / inputs)) takes parameters as [outputs, inputs]; those of
    this module's blocks are [inputs, outputs] (x @ w) and want ``inputs_first=True``."""

    _HOW = ("lr", "momentum", "nesterov", "weight_decay", "rms", "steps", "half", "inputs_first")

    def __init__(self, params, lr: float = 0.02, momentum: float = 0.95, nesterov: bool = True,
                 weight_decay: float = 0.0, rms: float | None = None, steps: int = 5,
                 half: bool | None = True, inputs_first: bool = False):
        super().__init__(params, dict(lr=lr, momentum=momentum, nesterov=nesterov,
                                      weight_decay=weight_decay, rms=rms, steps=steps, half=half,
                                      inputs_first=inputs_first))
        for group in self.param_groups:
            if any(p.dim() != 2 for p in group["params"]):
                raise ValueError("Muon takes matrices; give other parameters to another optimiser")

    def __setstate__(self, state):
        super().__setstate__(state)
        for group in self.param_groups:
            group.setdefault("inputs_first", False)  # (a checkpoint from before there was one)

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        for group in self.param_groups:
            places = {}
            for p in group["params"]:
                if p.grad is None or p.numel() == 0:
                    continue
                state = self.state[p]
                if "momentum" not in state:
                    state["momentum"] = torch.zeros_like(p, dtype=torch.float32)
                g = p.grad
                if g.stride() != p.stride():  # in the weight's order
                    g = torch.empty_like(p, dtype=g.dtype).copy_(g)
                for at, t in zip(places.setdefault(p.device, ([], [], [])),
                                 (p, g, state["momentum"])):
                    at.append(t)
            how = {k: group[k] for k in self._HOW}  # (schedules and users add keys of their own)
            for weights, grads, momenta in places.values():
                B.sparge_muon_step(weights, grads, momenta, **how)
        return loss

    def load_state_dict(self, state_dict):
        super().load_state_dict(state_dict)
        # (which casts a state to its parameter's type)
        mine = [p for group in self.param_groups for p in group["params"]]
        theirs = [i for group in state_dict["param_groups"] for i in group["params"]]
        for p, i in zip(mine, theirs):
            m = state_dict["state"].get(i, {}).get("momentum")
            if m is not None:
                self.state[p]["momentum"] = torch.empty_like(p, dtype=torch.float32).copy_(m)


def distillation_step(student, teacher, x: torch.Tensor, optimizer: torch.optim.Optimizer,
                      max_grad_norm: float | None = None, **inputs) -> float:
    """One fine-tuning step of the sparse student against the frozen dense
    teacher: loss = mean((student(x) - teacher(x))^2); backward through the
    library's sparse attention backward; gradients clipped to the global norm
    ``max_grad_norm`` where that is given; optimiser step. ``inputs`` (grid,
    modulation, context, kv_len) go to both. Returns the loss."""
    with torch.no_grad():
        target = teacher(x, **inputs)
    optimizer.zero_grad(set_to_none=True)
    loss = torch.mean((student(x, **inputs) - target) ** 2)
    loss.backward()
    if max_grad_norm is not None:
        clip_grad_norm_(student.parameters(), max_grad_norm)
    optimizer.step()
    return float(loss.item())
