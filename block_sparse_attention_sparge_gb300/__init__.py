"""GB300-native (sm_103a) SpargeAttention2 hot path.

Hybrid Top-k + Top-p block-mask construction from a mean-pooled attention map,
followed by block-sparse attention forward and backward that compute only the
kept tiles; and the operators around it in a transformer block (head layout
with norm and rotary positions, residual join with the next norm, gradient
clipping).  The work runs in the CUDA kernels of ``libsparge.so`` (C ABI in
``include/sparge.h``); ``binding`` marshals torch tensors to it.
"""

from .binding import (  # noqa: F401
    RopeAxes,
    SpargeError,
    load_library,
    sparge_attn_bwd,
    sparge_attn_fwd,
    sparge_clip_grads,
    sparge_cross_bwd,
    sparge_cross_fwd,
    sparge_debug_wait_probe,
    sparge_heads_bwd,
    sparge_heads_fwd,
    sparge_mask,
    sparge_mask_from_prob,
    sparge_muon_step,
    sparge_orthogonalize,
    sparge_pool,
    sparge_resnorm_bwd,
    sparge_resnorm_fwd,
)

__all__ = [
    "SpargeError",
    "load_library",
    "sparge_pool",
    "sparge_mask",
    "sparge_mask_from_prob",
    "sparge_attn_fwd",
    "sparge_attn_bwd",
    "RopeAxes",
    "sparge_heads_fwd",
    "sparge_heads_bwd",
    "sparge_resnorm_fwd",
    "sparge_resnorm_bwd",
    "sparge_clip_grads",
    "sparge_cross_fwd",
    "sparge_cross_bwd",
    "sparge_orthogonalize",
    "sparge_muon_step",
    "sparge_debug_wait_probe",
]
