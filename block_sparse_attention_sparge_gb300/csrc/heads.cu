// Query, key and value projections on their way to the attention and back:
// RMS norm of Q and K, rotary positions with up to three axes, the change from
// token-major [B, N, H, d] to the attention's head-major bf16 [B, H, N, d], and
// the gradients of all of it.
//
// Mathematics, for one token of Q or K with channels x (of one head, or of all
// heads when the norm spans the token):
//   r = 1 / sqrt(mean(x^2) + eps),  u = x * r * w
//   pair j of axis a turns by t_j = pos_a * f_j:
//   y_a = u_a cos t - u_b sin t,  y_b = u_a sin t + u_b cos t.
// Backward, g = the gradient turned by -t:
//   dw = sum over tokens of g * x * r,  q = g * w,
//   dx = r * q - x * r^3 * mean(q * x).
// Sums and products are fp32; y and dx are rounded once.
//
// A frequency is held as a 64-bit fraction of a turn (f / 2 pi * 2^64), so
// pos * f is reduced to one turn by the wrap of an integer product, exactly for
// every 32-bit position; sincospif then sees an argument in [-1, 1).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "rows.cuh"

namespace sparge {

namespace {

struct HeadsPart {
  const void* x;
  const void* w;
  void* y;  // head-major bf16: the result, or the gradient that comes back
  void* dx;
  float* dw_part;  // [slots][H * d]
  int64_t xs[3], ds[3];
  int C, W, plain;
};

struct HeadsParams {
  HeadsPart part[3];
  const int32_t* grid;
  const int32_t* pos;
  int64_t pos_ld;  // elements between samples of pos
  int M, N;        // rows in all, rows of one sample
  int norm, rotate, w_bf16;
  float eps;
  uint64_t turn[64];
  uint8_t axis[64];
};

// Cosines and sines of T tokens in shared memory: [T][D / 2].
template <int T, int D>
SPARGE_DEV void token_angles(const HeadsParams& p, const Slot& s, const uint64_t* turn,
                             const uint8_t* axis, int row0, float2* out) {
  constexpr int P = D / 2;
  for (int i = s.tid; i < T * P; i += s.W * 32) {
    const int j = i % P, row = row0 + i / P;
    int pos = 0;
    if (row < p.M) {
      const int b = row / p.N, n = row - b * p.N;
      const int a = axis[j];
      if (p.pos != nullptr) {
        pos = p.pos[b * p.pos_ld + static_cast<int64_t>(n) * 3 + a];
      } else {
        // Token n of a (t, h, w) grid; tokens behind it stay at position 0.
        const int t = p.grid[3 * b], h = p.grid[3 * b + 1], w = p.grid[3 * b + 2];
        if (t > 0 && h > 0 && w > 0) {
          const int64_t hw = static_cast<int64_t>(h) * w;
          const int it = hw > n ? 0 : n / static_cast<int>(hw);
          const int rest = n - static_cast<int>(it * hw);
          const int ih = rest / w;
          if (it < t) pos = a == 0 ? it : a == 1 ? ih : rest - ih * w;
        }
      }
    }
    const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * turn[j];
    const float half_turns =
        static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f;  // 2^-31
    float sn, cs;
    sincospif(half_turns, &sn, &cs);
    out[i] = make_float2(cs, sn);
  }
}

// This thread's eight channels of one token of a token-major tensor: eight in
// a row when pairs are adjacent, four and their four partners otherwise.
template <typename T, bool INTER, int D>
SPARGE_DEV Raw8<T> load_row(const T* p) {
  if constexpr (INTER)
    return load8(p);
  else
    return load4x2(p, p + D / 2);
}
template <typename T, bool INTER, int D>
SPARGE_DEV void store_row(T* p, const float (&f)[8]) {
  if constexpr (INTER)
    store8(p, f);
  else
    store4x2(p, p + D / 2, f);
}

// Turns the four pairs by (cos, sin); sgn = -1 turns them back.
template <bool INTER>
SPARGE_DEV void rotate8(float (&f)[8], const float4* cs, float sgn) {
  const float4 c0 = cs[0], c1 = cs[1];
  const float c[4] = {c0.x, c0.z, c1.x, c1.z};
  const float n[4] = {sgn * c0.y, sgn * c0.w, sgn * c1.y, sgn * c1.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int ia = INTER ? 2 * j : j, ib = INTER ? 2 * j + 1 : j + 4;
    const float a = f[ia], b = f[ib];
    f[ia] = a * c[j] - b * n[j];
    f[ib] = a * n[j] + b * c[j];
  }
}

// Sums over the lanes of one head (D / 8 of them, aligned).
template <int D, int K>
SPARGE_DEV void head_sum(float (&v)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  }
}

// The eight weights of this thread's channels (1 without a weight).
template <bool INTER, int D>
SPARGE_DEV void load_weight(const HeadsParams& p, const void* w, bool active, int c, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = 1.f;
  if (w == nullptr || !active) return;
  if (p.w_bf16)
    unpack8(load_row<__nv_bfloat16, INTER, D>(static_cast<const __nv_bfloat16*>(w) + c), f);
  else
    unpack8(load_row<float, INTER, D>(static_cast<const float*>(w) + c), f);
}

// What a thread keeps of its place: its head, and its first channel in it.
template <bool INTER, int D>
struct Place {
  bool active;
  int head, c;  // c: first channel within the head
  SPARGE_DEV Place(const Slot& s, int C) {
    constexpr int L = D / 8;  // threads of one head
    active = s.tid * 8 < C;
    head = s.tid / L;
    c = (s.tid % L) * (INTER ? 8 : 4);
  }
};

template <typename TX, bool INTER, int D, int T, int THREADS>
__global__ void __launch_bounds__(THREADS) heads_fwd_kernel(const __grid_constant__ HeadsParams p) {
  __shared__ float red[kSlotRedFloats];
  __shared__ __align__(16) float2 angles[kMaxSlots * 2 * T * 64];
  __shared__ uint64_t turn[64];
  __shared__ uint8_t axis[64];
  const HeadsPart& part = p.part[blockIdx.y];
  const bool rot = p.rotate && !part.plain;
  const int norm = part.plain ? 0 : p.norm;
  if (threadIdx.x < 64) {
    turn[threadIdx.x] = p.turn[threadIdx.x];
    axis[threadIdx.x] = p.axis[threadIdx.x];
  }
  __syncthreads();
  const int per_cta = slots_per_cta(part.W);
  Slot s = make_slot(part.W, red);
  if (s.index >= per_cta) return;
  const Place<INTER, D> at(s, part.C);
  const int wc = norm == 1 ? at.head * D + at.c : at.c;
  float w[8];
  load_weight<INTER, D>(p, norm ? part.w : nullptr, at.active, wc, w);

  const TX* x = static_cast<const TX*>(part.x) + at.head * part.xs[2] + at.c;
  const int H = part.C / D;
  __nv_bfloat16* y = static_cast<__nv_bfloat16*>(part.y) + static_cast<int64_t>(at.head) * p.N * D + at.c;
  const int nslots = gridDim.x * per_cta;
  float2* ang = angles + s.index * 2 * T * 64;
  int buf = 0;
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x * per_cta + s.index) * T; row0 < p.M;
       row0 += static_cast<int64_t>(nslots) * T, buf ^= 1) {
    Raw8<TX> raw[T];
    int b = static_cast<int>(row0) / p.N, n = static_cast<int>(row0) - b * p.N;
    int64_t yo[T];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const bool ok = at.active && row0 + t < p.M;
      raw[t] = ok ? load_row<TX, INTER, D>(x + b * part.xs[0] + n * part.xs[1]) : zero8<TX>();
      yo[t] = ok ? (static_cast<int64_t>(b) * H * p.N + n) * D : -1;
      if (++n == p.N) n = 0, ++b;
    }
    float2* cs = ang + buf * T * 64;
    if (rot) token_angles<T, D>(p, s, turn, axis, static_cast<int>(row0), cs);
    float v[T][8], ss[T];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      unpack8(raw[t], v[t]);
      ss[t] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss[t] += v[t][i] * v[t][i];
    }
    if (norm == 1 && s.W > 1) {
      slot_sum(s, ss);  // its barrier also publishes the angles
    } else {
      if (norm == 1) slot_sum(s, ss);
      if (norm == 2) head_sum<D>(ss);
      if (rot) slot_sync(s);
    }
    const float inv = 1.f / (norm == 1 ? part.C : D);
#pragma unroll
    for (int t = 0; t < T; ++t) {
      if (norm) {
        const float r = 1.f / sqrtf(ss[t] * inv + p.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[t][i] *= r * w[i];
      }
      if (rot)
        rotate8<INTER>(v[t], reinterpret_cast<const float4*>(
                                 cs + t * (D / 2) + (INTER ? at.c / 2 : at.c)), 1.f);
      if (yo[t] >= 0) store_row<__nv_bfloat16, INTER, D>(y + yo[t], v[t]);
    }
  }
}

template <typename TX, bool INTER, int D, int T, int THREADS>
__global__ void __launch_bounds__(THREADS) heads_bwd_kernel(const __grid_constant__ HeadsParams p) {
  __shared__ float red[kSlotRedFloats];
  __shared__ __align__(16) float2 angles[kMaxSlots * 2 * T * 64];
  __shared__ uint64_t turn[64];
  __shared__ uint8_t axis[64];
  grid_launch_dependents();
  const HeadsPart& part = p.part[blockIdx.y];
  const bool rot = p.rotate && !part.plain;
  const int norm = part.plain ? 0 : p.norm;
  if (threadIdx.x < 64) {
    turn[threadIdx.x] = p.turn[threadIdx.x];
    axis[threadIdx.x] = p.axis[threadIdx.x];
  }
  __syncthreads();
  const int per_cta = slots_per_cta(part.W);
  Slot s = make_slot(part.W, red);
  if (s.index >= per_cta) return;
  const Place<INTER, D> at(s, part.C);
  const int wc = norm == 1 ? at.head * D + at.c : at.c;
  float w[8], dw[8];
  load_weight<INTER, D>(p, norm ? part.w : nullptr, at.active, wc, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = 0.f;

  const TX* x = static_cast<const TX*>(part.x) + at.head * part.xs[2] + at.c;
  TX* dx = static_cast<TX*>(part.dx) + at.head * part.ds[2] + at.c;
  const int H = part.C / D;
  const __nv_bfloat16* dy = static_cast<const __nv_bfloat16*>(part.y) +
                            static_cast<int64_t>(at.head) * p.N * D + at.c;
  const int nslots = gridDim.x * per_cta;
  const int slot = blockIdx.x * per_cta + s.index;
  float2* ang = angles + s.index * 2 * T * 64;
  int buf = 0;
  for (int64_t row0 = static_cast<int64_t>(slot) * T; row0 < p.M;
       row0 += static_cast<int64_t>(nslots) * T, buf ^= 1) {
    Raw8<TX> raw[T];
    Raw8<__nv_bfloat16> rawg[T];
    int b = static_cast<int>(row0) / p.N, n = static_cast<int>(row0) - b * p.N;
    TX* out[T];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const bool ok = at.active && row0 + t < p.M;
      rawg[t] = ok ? load_row<__nv_bfloat16, INTER, D>(
                         dy + (static_cast<int64_t>(b) * H * p.N + n) * D)
                   : zero8<__nv_bfloat16>();
      raw[t] = ok && norm ? load_row<TX, INTER, D>(x + b * part.xs[0] + n * part.xs[1])
                          : zero8<TX>();
      out[t] = ok ? dx + b * part.ds[0] + n * part.ds[1] : nullptr;
      if (++n == p.N) n = 0, ++b;
    }
    const float2* cs = ang + buf * T * 64;
    if (rot) {
      token_angles<T, D>(p, s, turn, axis, static_cast<int>(row0), ang + buf * T * 64);
      slot_sync(s);
    }
    float g[T][8], v[T][8], sums[2 * T];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      unpack8(rawg[t], g[t]);
      if (rot)
        rotate8<INTER>(g[t], reinterpret_cast<const float4*>(
                                 cs + t * (D / 2) + (INTER ? at.c / 2 : at.c)), -1.f);
      if (norm) {
        unpack8(raw[t], v[t]);
        sums[2 * t] = sums[2 * t + 1] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sums[2 * t] += v[t][i] * v[t][i];
          sums[2 * t + 1] += v[t][i] * (g[t][i] * w[i]);
        }
      }
    }
    if (norm == 1) slot_sum(s, sums);
    if (norm == 2) head_sum<D>(sums);
    const float inv = 1.f / (norm == 1 ? part.C : D);
#pragma unroll
    for (int t = 0; t < T; ++t) {
      if (norm) {
        const float r = 1.f / sqrtf(sums[2 * t] * inv + p.eps);
        const float m = sums[2 * t + 1] * inv * r * r;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dw[i] += g[t][i] * (v[t][i] * r);
          g[t][i] = r * (g[t][i] * w[i] - v[t][i] * m);
        }
      }
      if (out[t] != nullptr) store_row<TX, INTER, D>(out[t], g[t]);
    }
  }
  if (norm && part.dw_part != nullptr && at.active)
    store_row<float, INTER, D>(
        part.dw_part + static_cast<int64_t>(slot) * part.C + at.head * D + at.c, dw);
}

// Slots of one part: a CTA per resident place of the machine, shared by the
// parts, and no more than there are row groups.
int heads_ctas(int M, int T, int n_parts, int per_cta, int per_sm) {
  const int64_t units = (static_cast<int64_t>(M) + T - 1) / T;
  const int64_t need = (units + per_cta - 1) / per_cta;
  const int64_t most = (kSMs * per_sm + n_parts - 1) / n_parts;
  return static_cast<int>(std::max<int64_t>(1, std::min(need, most)));
}

struct HeadsPlan {
  int ctas, threads, tier;
  int n;             // parts
  size_t dw_off[3];  // into the workspace
  size_t bytes;
};

HeadsPlan heads_plan(const sparge_heads& a, bool bwd) {
  HeadsPlan pl = {};
  int threads = 32, slots_min = kMaxSlots;
  pl.n = a.n_parts;
  for (int i = 0; i < a.n_parts; ++i) {
    const int W = slot_warps(a.part[i].H * a.d);
    threads = std::max(threads, W * slots_per_cta(W) * 32);
    slots_min = std::min(slots_min, slots_per_cta(W));
  }
  pl.threads = threads;
  pl.tier = tier_of(threads);
  const int per_sm = std::max(1, 1280 / threads);
  const int rows = bwd ? kTiers[pl.tier].bwd_rows : kTiers[pl.tier].fwd_rows;
  pl.ctas = heads_ctas(a.B * a.N, rows, a.n_parts, slots_min, per_sm);
  for (int i = 0; i < a.n_parts; ++i) {
    if (!bwd || a.norm == 0 || a.part[i].plain || a.part[i].dweight == nullptr) continue;
    const int C = a.part[i].H * a.d;
    pl.dw_off[i] = pl.bytes;
    pl.bytes += static_cast<size_t>(pl.ctas) * slots_per_cta(slot_warps(C)) * C * sizeof(float);
  }
  return pl;
}

HeadsParams heads_params(const sparge_heads& a) {
  HeadsParams p = {};
  for (int i = 0; i < a.n_parts; ++i) {
    const sparge_heads_part& s = a.part[i];
    HeadsPart& o = p.part[i];
    o.x = s.x;
    o.w = s.weight;
    o.y = s.y;
    o.dx = s.dx;
    for (int k = 0; k < 3; ++k) o.xs[k] = s.x_stride[k], o.ds[k] = s.dx_stride[k];
    o.C = s.H * a.d;
    o.W = slot_warps(o.C);
    o.plain = s.plain;
  }
  p.grid = a.grid;
  p.pos = a.pos;
  p.pos_ld = a.pos_batch == 1 ? 0 : static_cast<int64_t>(a.N) * 3;
  p.M = a.B * a.N;
  p.N = a.N;
  p.norm = a.norm;
  p.w_bf16 = a.weight_type == SPARGE_BF16;
  p.eps = a.eps;
  p.rotate = a.rope != nullptr;
  if (a.rope != nullptr) {
    for (int j = 0; j < a.d / 2; ++j) p.turn[j] = a.rope->turn[j], p.axis[j] = a.rope->axis[j];
  }
  return p;
}

template <typename TX, bool INTER, int D, int I>
void launch_tier(const HeadsParams& p, const HeadsPlan& pl, bool bwd, cudaStream_t st) {
  constexpr Tier t = kTiers[I];
  const dim3 grid(pl.ctas, pl.n);
  if (bwd)
    heads_bwd_kernel<TX, INTER, D, t.bwd_rows, t.threads><<<grid, pl.threads, 0, st>>>(p);
  else
    heads_fwd_kernel<TX, INTER, D, t.fwd_rows, t.threads><<<grid, pl.threads, 0, st>>>(p);
}

template <typename TX, bool INTER, int D>
cudaError_t launch_heads(const HeadsParams& p, const HeadsPlan& pl, bool bwd, cudaStream_t st) {
  if (pl.tier == 0) launch_tier<TX, INTER, D, 0>(p, pl, bwd, st);
  if (pl.tier == 1) launch_tier<TX, INTER, D, 1>(p, pl, bwd, st);
  if (pl.tier == 2) launch_tier<TX, INTER, D, 2>(p, pl, bwd, st);
  return cudaGetLastError();
}

cudaError_t dispatch_heads(const sparge_heads& a, const HeadsParams& p, const HeadsPlan& pl,
                           bool bwd, cudaStream_t st) {
  const bool inter = a.rope == nullptr || a.rope->interleaved;
  const int key = (a.x_type == SPARGE_F32) * 4 + inter * 2 + (a.d == 128);
  switch (key) {
    case 0: return launch_heads<__nv_bfloat16, false, 64>(p, pl, bwd, st);
    case 1: return launch_heads<__nv_bfloat16, false, 128>(p, pl, bwd, st);
    case 2: return launch_heads<__nv_bfloat16, true, 64>(p, pl, bwd, st);
    case 3: return launch_heads<__nv_bfloat16, true, 128>(p, pl, bwd, st);
    case 4: return launch_heads<float, false, 64>(p, pl, bwd, st);
    case 5: return launch_heads<float, false, 128>(p, pl, bwd, st);
    case 6: return launch_heads<float, true, 64>(p, pl, bwd, st);
    default: return launch_heads<float, true, 128>(p, pl, bwd, st);
  }
}

int check_aligned(const void* p, size_t to) {
  if (p == nullptr) return SPARGE_ERR_INVALID_ARG;
  return reinterpret_cast<uintptr_t>(p) % to == 0 ? SPARGE_OK : SPARGE_ERR_MISALIGNED;
}

#define HEADS_TRY(expr)               \
  do {                                \
    const int rc_ = (expr);           \
    if (rc_ != SPARGE_OK) return rc_; \
  } while (0)

// Strides in elements of a token-major tensor whose rows of a head are read in
// 16-byte pieces.
int check_strides(const int64_t (&s)[3], int x_type) {
  const int64_t step = x_type == SPARGE_F32 ? 4 : 8;
  for (int k = 0; k < 3; ++k) {
    if (s[k] < 0) return SPARGE_ERR_INVALID_ARG;
    if (s[k] % step != 0) return SPARGE_ERR_MISALIGNED;
  }
  return SPARGE_OK;
}

int check_heads(const sparge_heads* a, bool bwd) {
  if (a == nullptr) return SPARGE_ERR_INVALID_ARG;
  if (a->B < 1 || a->N < 1 || a->n_parts < 1 || a->n_parts > 3) return SPARGE_ERR_INVALID_ARG;
  if (static_cast<int64_t>(a->B) * a->N > INT32_MAX) return SPARGE_ERR_UNSUPPORTED;
  if (a->d != 64 && a->d != 128) return SPARGE_ERR_UNSUPPORTED;
  if (a->x_type != SPARGE_BF16 && a->x_type != SPARGE_F32) return SPARGE_ERR_UNSUPPORTED;
  if (a->weight_type != SPARGE_BF16 && a->weight_type != SPARGE_F32) return SPARGE_ERR_UNSUPPORTED;
  if (a->norm < SPARGE_HEADS_NORM_NONE || a->norm > SPARGE_HEADS_NORM_HEAD)
    return SPARGE_ERR_INVALID_ARG;
  if (!isfinite(a->eps) || a->eps < 0.f) return SPARGE_ERR_INVALID_ARG;
  if (a->rope != nullptr) {
    if (a->rope->d != a->d) return SPARGE_ERR_INVALID_ARG;
    for (int j = 0; j < a->d / 2; ++j)
      if (a->rope->axis[j] > 2) return SPARGE_ERR_INVALID_ARG;
    if ((a->grid == nullptr) == (a->pos == nullptr)) return SPARGE_ERR_INVALID_ARG;
    if (a->grid) HEADS_TRY(check_aligned(a->grid, 4));
    if (a->pos) {
      HEADS_TRY(check_aligned(a->pos, 4));
      if (a->pos_batch != 1 && a->pos_batch != a->B) return SPARGE_ERR_INVALID_ARG;
    }
  } else if (a->grid != nullptr || a->pos != nullptr) {
    return SPARGE_ERR_INVALID_ARG;
  }
  for (int i = 0; i < a->n_parts; ++i) {
    const sparge_heads_part& s = a->part[i];
    if (s.H < 1) return SPARGE_ERR_INVALID_ARG;
    if (s.H > kMaxRowChannels / a->d) return SPARGE_ERR_UNSUPPORTED;
    const bool normed = a->norm != SPARGE_HEADS_NORM_NONE && !s.plain;
    HEADS_TRY(check_aligned(s.y, 16));
    if (!bwd || normed) {
      HEADS_TRY(check_aligned(s.x, 16));
      HEADS_TRY(check_strides(s.x_stride, a->x_type));
    }
    if (normed && s.weight) HEADS_TRY(check_aligned(s.weight, 16));
    if (bwd) {
      HEADS_TRY(check_aligned(s.dx, 16));
      HEADS_TRY(check_strides(s.dx_stride, a->x_type));
      if (normed && s.dweight) HEADS_TRY(check_aligned(s.dweight, 4));
    }
  }
  return SPARGE_OK;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? SPARGE_OK : SPARGE_ERR_CUDA; }

}  // namespace

}  // namespace sparge

using namespace sparge;

extern "C" {

int sparge_rope_init(sparge_rope* rope, int32_t d, const int32_t* pairs, double theta,
                     const double* scale, int32_t interleaved) {
  if (rope == nullptr || pairs == nullptr) return SPARGE_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return SPARGE_ERR_UNSUPPORTED;
  if (!isfinite(theta) || theta <= 0.0) return SPARGE_ERR_INVALID_ARG;
  int total = 0;
  for (int a = 0; a < 3; ++a) {
    if (pairs[a] < 0 || pairs[a] > d / 2) return SPARGE_ERR_INVALID_ARG;
    total += pairs[a];
    if (scale != nullptr && !isfinite(scale[a])) return SPARGE_ERR_INVALID_ARG;
  }
  if (total > d / 2) return SPARGE_ERR_INVALID_ARG;
  sparge_rope r = {};
  r.d = d;
  r.interleaved = interleaved != 0;
  int j = 0;
  for (int a = 0; a < 3; ++a) {
    for (int i = 0; i < pairs[a]; ++i, ++j) {
      const double f = (scale ? scale[a] : 1.0) * pow(theta, -static_cast<double>(i) / pairs[a]);
      const double turns = f / 6.283185307179586476925;
      if (!isfinite(turns)) return SPARGE_ERR_INVALID_ARG;
      const double frac = turns - floor(turns);
      r.turn[j] = frac >= 1.0 ? 0 : static_cast<uint64_t>(ldexp(frac, 64));
      r.axis[j] = static_cast<uint8_t>(a);
    }
  }
  *rope = r;
  return SPARGE_OK;
}

int sparge_heads_fwd(const sparge_heads* args, sparge_stream_t stream) {
  HEADS_TRY(check_heads(args, false));
  return status_of(dispatch_heads(*args, heads_params(*args), heads_plan(*args, false), false,
                                  stream));
}

int sparge_heads_bwd_workspace_bytes(const sparge_heads* args, size_t* bytes) {
  if (bytes == nullptr) return SPARGE_ERR_INVALID_ARG;
  HEADS_TRY(check_heads(args, true));
  *bytes = heads_plan(*args, true).bytes;
  return SPARGE_OK;
}

int sparge_heads_bwd(const sparge_heads* args, void* workspace, size_t ws_bytes,
                     sparge_stream_t stream) {
  HEADS_TRY(check_heads(args, true));
  const HeadsPlan pl = heads_plan(*args, true);
  if (pl.bytes > 0) {
    if (workspace == nullptr || ws_bytes < pl.bytes) return SPARGE_ERR_WORKSPACE;
    HEADS_TRY(check_aligned(workspace, 16));
  }
  HeadsParams p = heads_params(*args);
  ReduceJobs jobs = {};
  for (int i = 0; i < args->n_parts; ++i) {
    const sparge_heads_part& s = args->part[i];
    if (args->norm == SPARGE_HEADS_NORM_NONE || s.plain || s.dweight == nullptr) continue;
    const int C = s.H * args->d;
    p.part[i].dw_part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + pl.dw_off[i]);
    // One row of C sums a slot; with a norm over each head, H rows of d.
    const bool token = args->norm == SPARGE_HEADS_NORM_TOKEN;
    ReduceJob& j = jobs.job[jobs.n++];
    j.src = p.part[i].dw_part;
    j.C = token ? C : args->d;
    j.ld = j.C;
    j.nrow = pl.ctas * slots_per_cta(slot_warps(C)) * (token ? 1 : s.H);
    j.nout = 1;
    j.out = s.dweight;
    j.out_bf16 = args->weight_type == SPARGE_BF16;
  }
  HEADS_TRY(status_of(dispatch_heads(*args, p, pl, true, stream)));
  if (jobs.n > 0) return status_of(launch_reduce_rows(jobs, stream));
  return SPARGE_OK;
}

}  // extern "C"
