// Entry points of the attention over a context: argument checks, workspace.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "cross.cuh"
#include "places.h"
#include "sparge.h"

namespace sparge {

namespace {

constexpr int kMaxTokens = 524288;
constexpr int64_t kMaxHeads = int64_t(1) << 20;       // B * H
constexpr int64_t kMaxTiles = (int64_t(1) << 31) - 1;  // of a grid

#define CROSS_TRY(expr)               \
  do {                                \
    const int rc_ = (expr);           \
    if (rc_ != SPARGE_OK) return rc_; \
  } while (0)

int check_sizes(const sparge_cross* a) {
  if (a == nullptr) return SPARGE_ERR_INVALID_ARG;
  if (a->B < 1 || a->H < 1 || a->Hk < 1 || a->N < 1 || a->M < 1 || a->d < 1)
    return SPARGE_ERR_INVALID_ARG;
  if ((a->Bk != 1 && a->Bk != a->B) || a->H % a->Hk != 0) return SPARGE_ERR_INVALID_ARG;
  if (!isfinite(a->softmax_scale * kLog2e)) return SPARGE_ERR_INVALID_ARG;  // (the exponents' factor)
  if (a->d != 64 && a->d != 128) return SPARGE_ERR_UNSUPPORTED;
  if (a->N > kMaxTokens || a->M > kMaxTokens) return SPARGE_ERR_UNSUPPORTED;
  const int64_t heads = static_cast<int64_t>(a->B) * a->H;
  const int64_t most = a->N > a->M ? a->N : a->M;
  if (heads > kMaxHeads || heads * ((most + 63) / 64) > kMaxTiles) return SPARGE_ERR_UNSUPPORTED;
  return SPARGE_OK;
}

int check_word(const void* p) {
  return reinterpret_cast<uintptr_t>(p) % 4 == 0 ? SPARGE_OK : SPARGE_ERR_MISALIGNED;
}

// A tensor [batch, heads, tokens, d] with strides in that order.
int check_heads_tensor(const void* p, const int64_t (&stride)[3], const int64_t (&n)[3]) {
  if (p == nullptr) return SPARGE_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return SPARGE_ERR_MISALIGNED;
  for (int k = 0; k < 3; ++k) {
    if (n[k] == 1) continue;
    if (stride[k] < 1) return SPARGE_ERR_INVALID_ARG;
    if (stride[k] % 8 != 0) return SPARGE_ERR_MISALIGNED;
    if (stride[k] >= int64_t(1) << 39) return SPARGE_ERR_UNSUPPORTED;  // TMA: 2^40 bytes
  }
  return SPARGE_OK;
}

struct Tensors {
  int64_t nq[3], nk[3], run;
  explicit Tensors(const sparge_cross& a)
      : nq{a.B, a.H, a.N}, nk{a.Bk, a.Hk, a.M}, run(a.d * 2) {}
  Layout at(const void* p, const int64_t (&stride)[3], bool keys) const {
    return layout_of(p, keys ? nk : nq, stride, run, 2);
  }
};

int check_cross(const sparge_cross* a, bool bwd) {
  CROSS_TRY(check_sizes(a));
  const Tensors t(*a);
  CROSS_TRY(check_heads_tensor(a->q, a->q_stride, t.nq));
  CROSS_TRY(check_heads_tensor(a->k, a->k_stride, t.nk));
  CROSS_TRY(check_heads_tensor(a->v, a->v_stride, t.nk));
  CROSS_TRY(check_heads_tensor(a->o, a->o_stride, t.nq));
  CROSS_TRY(check_word(a->kv_len));
  CROSS_TRY(check_word(a->lse));
  CROSS_TRY(check_word(a->status));
  Layout in[7] = {t.at(a->q, a->q_stride, false), t.at(a->k, a->k_stride, true),
                  t.at(a->v, a->v_stride, true)};
  Layout out[3];
  int n_in = 3, n_out = 0;
  auto words = [](const void* p, int64_t n) { return layout_of(p, {1, 1, 1}, {0, 0, 0}, 4 * n, 1); };
  if (a->kv_len != nullptr) in[n_in++] = words(a->kv_len, a->B);
  const Layout lse = words(a->lse, static_cast<int64_t>(a->B) * a->H * a->N);
  if (bwd) {
    if (a->lse == nullptr) return SPARGE_ERR_INVALID_ARG;
    CROSS_TRY(check_heads_tensor(a->dout, a->dout_stride, t.nq));
    CROSS_TRY(check_heads_tensor(a->dq, a->dq_stride, t.nq));
    CROSS_TRY(check_heads_tensor(a->dk, a->dk_stride, t.nk));
    CROSS_TRY(check_heads_tensor(a->dv, a->dv_stride, t.nk));
    in[n_in++] = t.at(a->o, a->o_stride, false);
    in[n_in++] = t.at(a->dout, a->dout_stride, false);
    in[n_in++] = lse;
    out[n_out++] = t.at(a->dq, a->dq_stride, false);
    out[n_out++] = t.at(a->dk, a->dk_stride, true);
    out[n_out++] = t.at(a->dv, a->dv_stride, true);
  } else {
    out[n_out++] = t.at(a->o, a->o_stride, false);
    if (a->lse != nullptr) out[n_out++] = lse;
  }
  for (int i = 0; i < n_out; ++i) {
    if (meets_itself(out[i])) return SPARGE_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (meet(out[i], out[j])) return SPARGE_ERR_INVALID_ARG;
    for (int j = 0; j < n_in; ++j)
      if (meet(out[i], in[j])) return SPARGE_ERR_INVALID_ARG;
  }
  return SPARGE_OK;
}

CrossGeom geom_of(const sparge_cross& a) {
  CrossGeom g = {a.B, a.Bk, a.H, a.Hk, a.N, a.M, a.d};
  g.group = a.H / a.Hk;
  g.Mq = (a.N + kCrossQ - 1) / kCrossQ;
  g.Mt = (a.M + kCrossK - 1) / kCrossK;
  g.scale = a.softmax_scale == 0.f ? 1.0f / sqrtf(static_cast<float>(a.d)) : a.softmax_scale;
  g.kv_len = a.kv_len;
  return g;
}

int check_workspace(const void* p, size_t have, size_t need) {
  if (need == 0) return SPARGE_OK;
  if (p == nullptr || have < need) return SPARGE_ERR_WORKSPACE;
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 ? SPARGE_OK : SPARGE_ERR_MISALIGNED;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? SPARGE_OK : SPARGE_ERR_CUDA; }

}  // namespace

}  // namespace sparge

using namespace sparge;

extern "C" {

int sparge_cross_fwd_workspace_bytes(const sparge_cross* args, size_t* bytes) {
  if (bytes == nullptr) return SPARGE_ERR_INVALID_ARG;
  CROSS_TRY(check_sizes(args));
  *bytes = cross_fwd_workspace_bytes(geom_of(*args));
  return SPARGE_OK;
}

int sparge_cross_fwd(const sparge_cross* args, void* workspace, size_t ws_bytes,
                     sparge_stream_t stream) {
  CROSS_TRY(check_cross(args, false));
  const CrossGeom g = geom_of(*args);
  CROSS_TRY(check_workspace(workspace, ws_bytes, cross_fwd_workspace_bytes(g)));
  return status_of(launch_cross_fwd(g, *args, workspace, stream));
}

int sparge_cross_bwd_workspace_bytes(const sparge_cross* args, size_t* bytes) {
  if (bytes == nullptr) return SPARGE_ERR_INVALID_ARG;
  CROSS_TRY(check_sizes(args));
  *bytes = cross_bwd_workspace_bytes(geom_of(*args));
  return SPARGE_OK;
}

int sparge_cross_bwd(const sparge_cross* args, void* workspace, size_t ws_bytes,
                     sparge_stream_t stream) {
  CROSS_TRY(check_cross(args, true));
  const CrossGeom g = geom_of(*args);
  CROSS_TRY(check_workspace(workspace, ws_bytes, cross_bwd_workspace_bytes(g)));
  return status_of(launch_cross_bwd(g, *args, workspace, stream));
}

}  // extern "C"
