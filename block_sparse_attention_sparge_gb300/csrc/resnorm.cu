// The residual join of one half-block and the norm that opens the next, in one
// pass over the rows, and its gradients.
//
// Mathematics, for one token (row) of C channels:
//   n = b                                  or  b * rb * post, rb = 1 / sqrt(mean(b^2) + eps)
//   y = x + gate * n
//   z = (y - mean) * rstd                  (mean 0 for the RMS norm)
//   h = z * gain + shift,                  gain = scale or 1 + scale
// Backward, from dy and dh, with mean, rstd and rb as the forward left them:
//   g = dh * gain,  d = dy + rstd * (g - mean(g) - z * mean(g * z))
//   dx = d,  dscale = sum dh * z,  dshift = sum dh,  dgate = sum d * n
//   db = d * gate                          or, with e = d * gate:
//   dpost = sum e * b * rb,  db = rb * (e * post - b * rb * mean(e * post * b * rb))
// y is recomputed from x and b, so it need not be kept.  All arithmetic is
// fp32; y, h, dx and db are rounded once when they are written.
//
// The variance is the sum of squares about each warp's own mean, joined by the
// exact rule for two groups, so a row whose mean is far above its spread keeps
// its digits.
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

struct ResnormParams {
  const void* x;
  const void* b;
  const float* gate;
  const float* scale;
  const float* shift;
  const float* post;
  void* y;
  void* h;
  float* stats;  // [3][M]: mean, rstd, rb
  const void* dy;
  const void* dh;
  void* dx;
  void* db;
  int64_t gate_ld, scale_ld, shift_ld;  // 0: one row for all groups
  int M, C, R;                          // rows, channels, rows of one group
  int norm, unit;
  int W;
  float eps, inv_c;
  // backward: column sums in the order gate, scale, shift, post
  float* sum[4];      // null: not wanted
  int by_group[4];    // written at the end of each item, else at the slot's end
  int items, parts, part_rows;  // items = groups * parts
};

template <typename T>
SPARGE_DEV void load_f32x8(const T* p, float (&f)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
  f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// Mean and sum of squares about it, of each of T rows, over the slot.  `cnt`
// channels of this warp are in use (a multiple of 8).
template <int T>
SPARGE_DEV void slot_moments(Slot& s, const float (&y)[T][8], bool active, int cnt, float inv_c,
                             float (&mean)[T], float (&m2)[T]) {
  const float inv = cnt > 0 ? 1.f / cnt : 0.f;
#pragma unroll
  for (int t = 0; t < T; ++t) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += y[t][i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    mean[t] = sum * inv;
    float sq = 0.f;
    if (active) {
#pragma unroll
      for (int i = 0; i < 8; ++i) sq += (y[t][i] - mean[t]) * (y[t][i] - mean[t]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    m2[t] = sq;
  }
  if (s.W == 1) return;
  static_assert(2 * T <= kSlotRed, "reduction buffer");
  float* red = s.red + s.phase * s.W * kSlotRed;
  s.phase ^= 1;
  if (s.lane == 0) {
#pragma unroll
    for (int t = 0; t < T; ++t) {
      red[s.warp * kSlotRed + 2 * t] = mean[t];
      red[s.warp * kSlotRed + 2 * t + 1] = m2[t];
    }
  }
  slot_sync(s);
  // Every warp but the last has 256 channels.
  const int last = static_cast<int>(1.f / inv_c + 0.5f) - (s.W - 1) * 256;
#pragma unroll
  for (int t = 0; t < T; ++t) mean[t] = m2[t] = 0.f;
  for (int w = 0; w < s.W; ++w) {
    const float n = w + 1 < s.W ? 256.f : static_cast<float>(last);
#pragma unroll
    for (int t = 0; t < T; ++t) mean[t] += n * red[w * kSlotRed + 2 * t];
  }
#pragma unroll
  for (int t = 0; t < T; ++t) mean[t] *= inv_c;
  for (int w = 0; w < s.W; ++w) {
    const float n = w + 1 < s.W ? 256.f : static_cast<float>(last);
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const float d = red[w * kSlotRed + 2 * t] - mean[t];
      m2[t] += red[w * kSlotRed + 2 * t + 1] + n * d * d;
    }
  }
}

template <typename TX, typename TB, int T, int THREADS>
__global__ void __launch_bounds__(THREADS) resnorm_fwd_kernel(
    const __grid_constant__ ResnormParams p) {
  __shared__ float red[kSlotRedFloats];
  Slot s = make_slot(p.W, red);
  const int per_cta = slots_per_cta(p.W);
  if (s.index >= per_cta) return;
  const int c = s.tid * 8;
  const bool active = c < p.C;
  const int cnt = max(0, min(256, p.C - s.warp * 256));
  const TX* x = static_cast<const TX*>(p.x) + c;
  const TB* b = static_cast<const TB*>(p.b) + c;
  TX* y_out = static_cast<TX*>(p.y) + c;
  TB* h_out = static_cast<TB*>(p.h) + c;

  float gate[8], gain[8], shift[8], post[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) gate[i] = gain[i] = post[i] = 1.f, shift[i] = 0.f;
  if (p.post != nullptr && active) load_f32x8(p.post + c, post);

  const int units_per_group = (p.R + T - 1) / T;
  const int units = (p.M / p.R) * units_per_group;
  const int nslots = gridDim.x * per_cta;
  int group = -1;
  for (int u = blockIdx.x * per_cta + s.index; u < units; u += nslots) {
    const int g = u / units_per_group, first = (u - g * units_per_group) * T;
    const int rows = min(T, p.R - first);
    const int64_t row0 = static_cast<int64_t>(g) * p.R + first;
    Raw8<TX> rx[T];
    Raw8<TB> rb[T];
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const bool ok = active && t < rows;
      rx[t] = ok ? load8(x + (row0 + t) * p.C) : zero8<TX>();
      rb[t] = ok && p.b != nullptr ? load8(b + (row0 + t) * p.C) : zero8<TB>();
    }
    if (g != group) {
      if (active && p.gate != nullptr && (group < 0 || p.gate_ld != 0))
        load_f32x8(p.gate + g * p.gate_ld + c, gate);
      if (active && p.scale != nullptr && (group < 0 || p.scale_ld != 0)) {
        load_f32x8(p.scale + g * p.scale_ld + c, gain);
        if (p.unit) {
#pragma unroll
          for (int i = 0; i < 8; ++i) gain[i] += 1.f;
        }
      }
      if (active && p.shift != nullptr && (group < 0 || p.shift_ld != 0))
        load_f32x8(p.shift + g * p.shift_ld + c, shift);
      group = g;
    }
    float y[T][8];
    float rbs[T];
    if (p.b != nullptr) {
#pragma unroll
      for (int t = 0; t < T; ++t) unpack8(rb[t], y[t]);
      if (p.post != nullptr) {
#pragma unroll
        for (int t = 0; t < T; ++t) {
          rbs[t] = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) rbs[t] += y[t][i] * y[t][i];
        }
        slot_sum(s, rbs);
#pragma unroll
        for (int t = 0; t < T; ++t) {
          rbs[t] = 1.f / sqrtf(rbs[t] * p.inv_c + p.eps);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[t][i] *= rbs[t] * post[i];
        }
      }
#pragma unroll
      for (int t = 0; t < T; ++t) {
        float xv[8];
        unpack8(rx[t], xv);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[t][i] = fmaf(gate[i], y[t][i], xv[i]);
        if (active && t < rows) store8(y_out + (row0 + t) * p.C, y[t]);
      }
    } else {
#pragma unroll
      for (int t = 0; t < T; ++t) unpack8(rx[t], y[t]);
    }
    float mean[T], sq[T];
    if (p.norm == SPARGE_NORM_LAYER) {
      slot_moments(s, y, active, cnt, p.inv_c, mean, sq);
    } else if (p.norm == SPARGE_NORM_RMS) {
#pragma unroll
      for (int t = 0; t < T; ++t) {
        mean[t] = sq[t] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sq[t] += y[t][i] * y[t][i];
      }
      slot_sum(s, sq);
    }
#pragma unroll
    for (int t = 0; t < T; ++t) {
      float rstd = 0.f;
      if (p.norm != SPARGE_NORM_NONE) {
        rstd = 1.f / sqrtf(sq[t] * p.inv_c + p.eps);
        float h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = fmaf((y[t][i] - mean[t]) * rstd, gain[i], shift[i]);
        if (active && t < rows) store8(h_out + (row0 + t) * p.C, h);
      }
      if (s.tid == 0 && t < rows && p.stats != nullptr) {
        if (p.norm != SPARGE_NORM_NONE) {
          p.stats[row0 + t] = mean[t];
          p.stats[p.M + row0 + t] = rstd;
        }
        if (p.post != nullptr) p.stats[2 * static_cast<int64_t>(p.M) + row0 + t] = rbs[t];
      }
    }
  }
}

template <typename TX, typename TB, int T, int THREADS>
__global__ void __launch_bounds__(THREADS) resnorm_bwd_kernel(
    const __grid_constant__ ResnormParams p) {
  __shared__ float red[kSlotRedFloats];
  grid_launch_dependents();
  Slot s = make_slot(p.W, red);
  const int per_cta = slots_per_cta(p.W);
  if (s.index >= per_cta) return;
  const int c = s.tid * 8;
  const bool active = c < p.C;
  const TX* x = static_cast<const TX*>(p.x) + c;
  const TB* b = static_cast<const TB*>(p.b) + c;
  const TX* dy = static_cast<const TX*>(p.dy) + c;
  const TB* dh = static_cast<const TB*>(p.dh) + c;
  TX* dx = static_cast<TX*>(p.dx) + c;
  TB* db = static_cast<TB*>(p.db) + c;

  float gate[8], gain[8], post[8], acc[4][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    gate[i] = gain[i] = post[i] = 1.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k][i] = 0.f;
  }
  if (p.post != nullptr && active) load_f32x8(p.post + c, post);

  const int nslots = gridDim.x * per_cta, slot = blockIdx.x * per_cta + s.index;
  bool first_item = true;
  for (int item = slot; item < p.items; item += nslots) {
    const int g = item / p.parts, part = item - g * p.parts;
    const int begin = min(p.R, part * p.part_rows), end = min(p.R, begin + p.part_rows);
    if (active && p.gate != nullptr && (first_item || p.gate_ld != 0))
      load_f32x8(p.gate + g * p.gate_ld + c, gate);
    if (active && p.scale != nullptr && (first_item || p.scale_ld != 0)) {
      load_f32x8(p.scale + g * p.scale_ld + c, gain);
      if (p.unit) {
#pragma unroll
        for (int i = 0; i < 8; ++i) gain[i] += 1.f;
      }
    }
    first_item = false;
    for (int first = begin; first < end; first += T) {
      const int rows = min(T, end - first);
      const int64_t row0 = static_cast<int64_t>(g) * p.R + first;
      Raw8<TX> rx[T], rdy[T];
      Raw8<TB> rb[T], rdh[T];
      float mean[T], rstd[T], rbs[T];
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const bool ok = active && t < rows;
        const int64_t at = (row0 + t) * p.C;
        rx[t] = ok && p.norm ? load8(x + at) : zero8<TX>();
        rb[t] = ok && p.b != nullptr ? load8(b + at) : zero8<TB>();
        rdy[t] = ok && p.dy != nullptr ? load8(dy + at) : zero8<TX>();
        rdh[t] = ok && p.dh != nullptr ? load8(dh + at) : zero8<TB>();
        mean[t] = rstd[t] = rbs[t] = 0.f;
        if (t < rows) {
          if (p.norm == SPARGE_NORM_LAYER) mean[t] = p.stats[row0 + t];
          if (p.norm) rstd[t] = p.stats[p.M + row0 + t];
          if (p.post != nullptr) rbs[t] = p.stats[2 * static_cast<int64_t>(p.M) + row0 + t];
        }
      }
      float z[T][8], d[T][8], sums[2 * T];
#pragma unroll
      for (int t = 0; t < T; ++t) {
        float n[8], q[8];
        unpack8(rx[t], z[t]);
        unpack8(rb[t], n);
        unpack8(rdh[t], q);
        const float scale_b = p.post != nullptr ? rbs[t] : 1.f;
        sums[2 * t] = sums[2 * t + 1] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float y = p.b != nullptr ? fmaf(gate[i], n[i] * (scale_b * post[i]), z[t][i]) : z[t][i];
          z[t][i] = p.norm ? (y - mean[t]) * rstd[t] : 0.f;
          d[t][i] = q[i] * gain[i];
          acc[1][i] += q[i] * z[t][i];
          acc[2][i] += q[i];
          sums[2 * t] += d[t][i];
          sums[2 * t + 1] += d[t][i] * z[t][i];
        }
      }
      if (p.norm) slot_sum(s, sums);
      float e[T];
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const float c1 = p.norm == SPARGE_NORM_LAYER ? sums[2 * t] * p.inv_c : 0.f;
        const float c2 = sums[2 * t + 1] * p.inv_c;
        float v[8];
        unpack8(rdy[t], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[t][i] = fmaf(rstd[t], d[t][i] - c1 - z[t][i] * c2, v[i]);
        if (active && t < rows) store8(dx + (row0 + t) * p.C, d[t]);
        if (p.b != nullptr) {
          unpack8(rb[t], v);
          e[t] = 0.f;
          if (p.post != nullptr) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float bh = v[i] * rbs[t];
              acc[0][i] += d[t][i] * (bh * post[i]);
              const float en = d[t][i] * gate[i];
              acc[3][i] += en * bh;
              d[t][i] = en * post[i];
              e[t] += d[t][i] * bh;
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              acc[0][i] += d[t][i] * v[i];
              d[t][i] *= gate[i];
            }
            if (active && t < rows) store8(db + (row0 + t) * p.C, d[t]);
          }
        }
      }
      if (p.post != nullptr) {
        slot_sum(s, e);
#pragma unroll
        for (int t = 0; t < T; ++t) {
          float v[8];
          unpack8(rb[t], v);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            d[t][i] = rbs[t] * (d[t][i] - v[i] * rbs[t] * (e[t] * p.inv_c));
          if (active && t < rows) store8(db + (row0 + t) * p.C, d[t]);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (!p.by_group[k]) continue;
      if (active && p.sum[k] != nullptr)
        store8(p.sum[k] + static_cast<int64_t>(item) * p.C + c, acc[k]);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[k][i] = 0.f;
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (!p.by_group[k] && active && p.sum[k] != nullptr)
      store8(p.sum[k] + static_cast<int64_t>(slot) * p.C + c, acc[k]);
  }
}

struct ResnormPlan {
  int W, per_cta, threads, ctas, slots;
  int tier;
  int groups, R;
  int items, parts, part_rows;
  // backward: a sum is written per item straight to the output (one part a
  // group), per item to the workspace, or per slot to the workspace
  bool wanted[4], by_group[4];
  size_t off[4], bytes;
};

ResnormPlan resnorm_plan(const sparge_resnorm& a, bool bwd) {
  ResnormPlan pl = {};
  const int64_t M = a.rows;
  pl.W = slot_warps(a.C);
  pl.per_cta = slots_per_cta(pl.W);
  pl.threads = pl.W * pl.per_cta * 32;
  pl.tier = tier_of(pl.threads);
  int groups = 1;
  if (a.gate) groups = std::max(groups, a.gate_groups);
  if (a.scale) groups = std::max(groups, a.scale_groups);
  if (a.shift) groups = std::max(groups, a.shift_groups);
  pl.groups = groups;
  pl.R = static_cast<int>(M / groups);
  const int T = bwd ? kTiers[pl.tier].bwd_rows : kTiers[pl.tier].fwd_rows;
  const int per_sm = std::max(1, 1024 / pl.threads);
  const int64_t most = static_cast<int64_t>(kSMs) * per_sm;
  if (!bwd) {
    const int64_t units = static_cast<int64_t>(groups) * ((pl.R + T - 1) / T);
    pl.ctas = static_cast<int>(std::max<int64_t>(
        1, std::min<int64_t>(most, (units + pl.per_cta - 1) / pl.per_cta)));
    return pl;
  }
  const int64_t target = most * pl.per_cta;  // slots that fill the machine
  const int64_t units = (pl.R + T - 1) / T;
  int64_t parts = std::max<int64_t>(1, std::min<int64_t>(units, target / groups));
  pl.part_rows = static_cast<int>((units + parts - 1) / parts) * T;
  pl.parts = (pl.R + pl.part_rows - 1) / pl.part_rows;
  pl.items = groups * pl.parts;
  pl.ctas = static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>(most, (static_cast<int64_t>(pl.items) + pl.per_cta - 1) / pl.per_cta)));
  pl.slots = pl.ctas * pl.per_cta;
  const void* const out[4] = {a.dgate, a.dscale, a.dshift, a.dpost};
  const int out_groups[4] = {a.gate_groups, a.scale_groups, a.shift_groups, 1};
  for (int k = 0; k < 4; ++k) {
    pl.wanted[k] = out[k] != nullptr;
    if (!pl.wanted[k]) continue;
    pl.by_group[k] = out_groups[k] > 1;
    if (pl.by_group[k] && pl.parts == 1) continue;
    const size_t rows = pl.by_group[k] ? pl.items : pl.slots;
    pl.off[k] = pl.bytes;
    pl.bytes += rows * a.C * sizeof(float);
  }
  return pl;
}

ResnormParams resnorm_params(const sparge_resnorm& a, const ResnormPlan& pl, bool bwd) {
  ResnormParams p = {};
  p.x = a.x;
  p.b = a.branch;
  p.gate = a.gate;
  p.scale = a.scale;
  p.shift = a.shift;
  p.post = a.post_weight;
  p.y = a.y;
  p.h = a.h;
  p.stats = a.stats;
  p.dy = a.dy;
  p.dh = a.dh;
  p.dx = a.dx;
  p.db = a.dbranch;
  p.gate_ld = a.gate_groups > 1 ? a.gate_stride : 0;
  p.scale_ld = a.scale_groups > 1 ? a.scale_stride : 0;
  p.shift_ld = a.shift_groups > 1 ? a.shift_stride : 0;
  p.M = static_cast<int>(a.rows);
  p.C = a.C;
  p.R = pl.R;
  // Without dh no gradient passes the norm: the backward is that of the join.
  p.norm = bwd && a.dh == nullptr ? SPARGE_NORM_NONE : a.norm;
  p.unit = a.unit_offset;
  p.W = pl.W;
  p.eps = a.eps;
  p.inv_c = 1.f / a.C;
  p.items = pl.items;
  p.parts = pl.parts;
  p.part_rows = pl.part_rows;
  return p;
}

template <typename TX, typename TB, int I>
void launch_tier(const ResnormParams& p, const ResnormPlan& pl, bool bwd, cudaStream_t st) {
  constexpr Tier t = kTiers[I];
  if (bwd)
    resnorm_bwd_kernel<TX, TB, t.bwd_rows, t.threads><<<pl.ctas, pl.threads, 0, st>>>(p);
  else
    resnorm_fwd_kernel<TX, TB, t.fwd_rows, t.threads><<<pl.ctas, pl.threads, 0, st>>>(p);
}

template <typename TX, typename TB>
cudaError_t launch_resnorm(const ResnormParams& p, const ResnormPlan& pl, bool bwd,
                           cudaStream_t st) {
  if (pl.tier == 0) launch_tier<TX, TB, 0>(p, pl, bwd, st);
  if (pl.tier == 1) launch_tier<TX, TB, 1>(p, pl, bwd, st);
  if (pl.tier == 2) launch_tier<TX, TB, 2>(p, pl, bwd, st);
  return cudaGetLastError();
}

cudaError_t dispatch_resnorm(const sparge_resnorm& a, const ResnormParams& p,
                             const ResnormPlan& pl, bool bwd, cudaStream_t st) {
  if (a.x_type == SPARGE_BF16)
    return launch_resnorm<__nv_bfloat16, __nv_bfloat16>(p, pl, bwd, st);
  if (a.branch_type == SPARGE_BF16) return launch_resnorm<float, __nv_bfloat16>(p, pl, bwd, st);
  return launch_resnorm<float, float>(p, pl, bwd, st);
}

int check_aligned(const void* p, size_t to) {
  if (p == nullptr) return SPARGE_ERR_INVALID_ARG;
  return reinterpret_cast<uintptr_t>(p) % to == 0 ? SPARGE_OK : SPARGE_ERR_MISALIGNED;
}

#define RESNORM_TRY(expr)             \
  do {                                \
    const int rc_ = (expr);           \
    if (rc_ != SPARGE_OK) return rc_; \
  } while (0)

int check_mod(const float* m, int32_t groups, int64_t stride, int64_t rows) {
  if (m == nullptr) return SPARGE_OK;
  RESNORM_TRY(check_aligned(m, 16));
  if (groups < 1 || rows % groups != 0) return SPARGE_ERR_INVALID_ARG;
  if (groups > 1) {
    if (stride < 0) return SPARGE_ERR_INVALID_ARG;
    if (stride % 4 != 0) return SPARGE_ERR_MISALIGNED;
  }
  return SPARGE_OK;
}

int check_resnorm(const sparge_resnorm* a, bool bwd) {
  if (a == nullptr) return SPARGE_ERR_INVALID_ARG;
  if (a->rows < 1 || a->C < 1) return SPARGE_ERR_INVALID_ARG;
  if (a->rows > INT32_MAX / 2 || a->C % 8 != 0 || a->C > kMaxRowChannels)
    return SPARGE_ERR_UNSUPPORTED;
  const bool types = (a->x_type == SPARGE_BF16 && a->branch_type == SPARGE_BF16) ||
                     (a->x_type == SPARGE_F32 &&
                      (a->branch_type == SPARGE_BF16 || a->branch_type == SPARGE_F32));
  if (!types) return SPARGE_ERR_UNSUPPORTED;
  if (a->norm < SPARGE_NORM_NONE || a->norm > SPARGE_NORM_RMS) return SPARGE_ERR_INVALID_ARG;
  if (!isfinite(a->eps) || a->eps < 0.f) return SPARGE_ERR_INVALID_ARG;
  const bool normed = a->norm != SPARGE_NORM_NONE;
  if (!normed && a->branch == nullptr) return SPARGE_ERR_INVALID_ARG;  // nothing to do
  if (!normed && (a->scale != nullptr || a->shift != nullptr)) return SPARGE_ERR_INVALID_ARG;
  if (a->branch == nullptr && (a->gate != nullptr || a->post_weight != nullptr))
    return SPARGE_ERR_INVALID_ARG;
  RESNORM_TRY(check_mod(a->gate, a->gate_groups, a->gate_stride, a->rows));
  RESNORM_TRY(check_mod(a->scale, a->scale_groups, a->scale_stride, a->rows));
  RESNORM_TRY(check_mod(a->shift, a->shift_groups, a->shift_stride, a->rows));
  // One row for all tokens, or the same rows as the others.
  int groups = 1;
  const float* const mods[3] = {a->gate, a->scale, a->shift};
  const int32_t counts[3] = {a->gate_groups, a->scale_groups, a->shift_groups};
  for (int k = 0; k < 3; ++k) {
    if (mods[k] == nullptr || counts[k] == 1) continue;
    if (groups != 1 && groups != counts[k]) return SPARGE_ERR_UNSUPPORTED;
    groups = counts[k];
  }
  if (a->branch) RESNORM_TRY(check_aligned(a->branch, 16));
  if (a->post_weight) RESNORM_TRY(check_aligned(a->post_weight, 16));
  if (!bwd || normed) RESNORM_TRY(check_aligned(a->x, 16));
  if (!bwd) {
    if (a->branch) RESNORM_TRY(check_aligned(a->y, 16));
    if (normed) RESNORM_TRY(check_aligned(a->h, 16));
    if (a->stats) RESNORM_TRY(check_aligned(a->stats, 4));
    return SPARGE_OK;
  }
  if (normed || a->post_weight != nullptr) RESNORM_TRY(check_aligned(a->stats, 4));
  if (a->dy == nullptr && a->dh == nullptr) return SPARGE_ERR_INVALID_ARG;
  if (!normed && a->dh != nullptr) return SPARGE_ERR_INVALID_ARG;
  if (a->dy) RESNORM_TRY(check_aligned(a->dy, 16));
  if (a->dh) RESNORM_TRY(check_aligned(a->dh, 16));
  RESNORM_TRY(check_aligned(a->dx, 16));
  if (a->branch) RESNORM_TRY(check_aligned(a->dbranch, 16));
  const void* const of[4] = {a->gate, a->scale, a->shift, a->post_weight};
  void* const sums[4] = {a->dgate, a->dscale, a->dshift, a->dpost};
  for (int k = 0; k < 4; ++k) {
    if (sums[k] == nullptr) continue;
    if (of[k] == nullptr) return SPARGE_ERR_INVALID_ARG;
    RESNORM_TRY(check_aligned(sums[k], 16));
  }
  return SPARGE_OK;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? SPARGE_OK : SPARGE_ERR_CUDA; }

}  // namespace

}  // namespace sparge

using namespace sparge;

extern "C" {

int sparge_resnorm_fwd(const sparge_resnorm* args, sparge_stream_t stream) {
  RESNORM_TRY(check_resnorm(args, false));
  const ResnormPlan pl = resnorm_plan(*args, false);
  return status_of(dispatch_resnorm(*args, resnorm_params(*args, pl, false), pl, false, stream));
}

int sparge_resnorm_bwd_workspace_bytes(const sparge_resnorm* args, size_t* bytes) {
  if (bytes == nullptr) return SPARGE_ERR_INVALID_ARG;
  RESNORM_TRY(check_resnorm(args, true));
  *bytes = resnorm_plan(*args, true).bytes;
  return SPARGE_OK;
}

int sparge_resnorm_bwd(const sparge_resnorm* args, void* workspace, size_t ws_bytes,
                       sparge_stream_t stream) {
  RESNORM_TRY(check_resnorm(args, true));
  const ResnormPlan pl = resnorm_plan(*args, true);
  if (pl.bytes > 0) {
    if (workspace == nullptr || ws_bytes < pl.bytes) return SPARGE_ERR_WORKSPACE;
    RESNORM_TRY(check_aligned(workspace, 16));
  }
  ResnormParams p = resnorm_params(*args, pl, true);
  float* const out[4] = {args->dgate, args->dscale, args->dshift, args->dpost};
  const int32_t groups[4] = {args->gate_groups, args->scale_groups, args->shift_groups, 1};
  ReduceJobs jobs = {};
  for (int k = 0; k < 4; ++k) {
    if (!pl.wanted[k]) continue;
    p.by_group[k] = pl.by_group[k];
    if (pl.by_group[k] && pl.parts == 1) {
      p.sum[k] = out[k];
      continue;
    }
    p.sum[k] = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + pl.off[k]);
    ReduceJob& j = jobs.job[jobs.n++];
    j.src = p.sum[k];
    j.out = out[k];
    j.C = args->C;
    j.ld = args->C;
    j.nout = pl.by_group[k] ? groups[k] : 1;
    j.nrow = pl.by_group[k] ? pl.parts : pl.slots;
    j.out_bf16 = 0;
  }
  RESNORM_TRY(status_of(dispatch_resnorm(*args, p, pl, true, stream)));
  if (jobs.n > 0) return status_of(launch_reduce_rows(jobs, stream));
  return SPARGE_OK;
}

}  // extern "C"
