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
//
// Bound by memory: the forward reads x and b and writes y and h, the backward
// reads x, b, dy and dh and writes dx and db, each value once; the statistics
// and the column sums stay in registers.  A slot of warps holds whole rows,
// because both norms need all of a row before its first value can be written.
// Measured: 32760 rows of 1536 (fp32 x, bf16 b): forward 93 us for 604 MB (6.5
// TB/s), backward 139 us for 906 MB (6.5 TB/s); bf16 with a norm before and after
// and one modulation a frame, backward: 104 us for 605 MB (5.8 TB/s, held back by
// instruction issue); 75600 rows of 5120, forward 472 us for 3.10 GB (6.6 TB/s),
// backward with fp32 x 1060 us for 7.0 GB (6.6 TB/s).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "common.cuh"
#include "rows.cuh"
#include "sparge.h"

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
  int items, parts;  // items = groups * parts
};

// Eight channels as packed pairs: every elementwise step is a packed operation.
struct F8 {
  uint64_t v[4];
};
SPARGE_DEV F8 f8(const float (&f)[8]) {
  return {{f32x2(f[0], f[1]), f32x2(f[2], f[3]), f32x2(f[4], f[5]), f32x2(f[6], f[7])}};
}
SPARGE_DEV F8 f8(float f) {
  const uint64_t u = f32x2(f, f);
  return {{u, u, u, u}};
}
SPARGE_DEV F8 fma(const F8& a, const F8& b, const F8& c) {
  return {{ffma2(a.v[0], b.v[0], c.v[0]), ffma2(a.v[1], b.v[1], c.v[1]),
           ffma2(a.v[2], b.v[2], c.v[2]), ffma2(a.v[3], b.v[3], c.v[3])}};
}
SPARGE_DEV F8 mul(const F8& a, const F8& b) {
  return {{fmul2(a.v[0], b.v[0]), fmul2(a.v[1], b.v[1]), fmul2(a.v[2], b.v[2]),
           fmul2(a.v[3], b.v[3])}};
}
SPARGE_DEV F8 add(const F8& a, const F8& b) {
  return {{fadd2(a.v[0], b.v[0]), fadd2(a.v[1], b.v[1]), fadd2(a.v[2], b.v[2]),
           fadd2(a.v[3], b.v[3])}};
}
SPARGE_DEV float total(const F8& a) {
  const uint64_t s = fadd2(fadd2(a.v[0], a.v[1]), fadd2(a.v[2], a.v[3]));
  return f32x2_lo(s) + f32x2_hi(s);
}
SPARGE_DEV float dot(const F8& a, const F8& b) {
  const uint64_t s = fadd2(ffma2(a.v[0], b.v[0], fmul2(a.v[1], b.v[1])),
                           ffma2(a.v[2], b.v[2], fmul2(a.v[3], b.v[3])));
  return f32x2_lo(s) + f32x2_hi(s);
}
SPARGE_DEV F8 f8(const Raw8<float>& r) {
  return {{f32x2(__uint_as_float(r.v[0].x), __uint_as_float(r.v[0].y)),
           f32x2(__uint_as_float(r.v[0].z), __uint_as_float(r.v[0].w)),
           f32x2(__uint_as_float(r.v[1].x), __uint_as_float(r.v[1].y)),
           f32x2(__uint_as_float(r.v[1].z), __uint_as_float(r.v[1].w))}};
}
SPARGE_DEV F8 f8(const Raw8<__nv_bfloat16>& r) {
  float f[8];
  unpack8(r, f);
  return f8(f);
}
template <typename T>
SPARGE_DEV F8 unstage(Ring src) {
  return f8(unstage8<T>(src));
}

// Eight channels of a thread are two fours: side by side when every tensor is
// bf16, 128 channels apart (32 lanes on) when one is fp32, so that a warp reads
// and writes whole sectors of it.
template <typename TX>
constexpr int four_step() {
  return sizeof(TX) == 2 ? 4 : 128;
}
template <int F, typename T>
SPARGE_DEV void stage_fours(Ring dst, const T* p, bool lo, bool hi) {
  if constexpr (F == 4) {
    if (lo) stage8(dst, p);
  } else if constexpr (sizeof(T) == 4) {
    if (lo) cp_async16(&dst[0], p);
    if (hi) cp_async16(&dst[1], p + F);
  } else {
    if (lo) cp_async8(&dst[0], p);
    if (hi) cp_async8(reinterpret_cast<uint2*>(&dst[0]) + 1, p + F);
  }
}
template <int F, typename T>
SPARGE_DEV void put(T* p, const F8& a, bool lo, bool hi) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[2 * i] = f32x2_lo(a.v[i]), f[2 * i + 1] = f32x2_hi(a.v[i]);
  const Raw8<T> r = pack8(f, T());
  if constexpr (F == 4) {
    if (lo) store_raw8(p, r);
  } else if constexpr (sizeof(T) == 4) {
    if (lo) *reinterpret_cast<uint4*>(p) = r.v[0];
    if (hi) *reinterpret_cast<uint4*>(p + F) = r.v[1];
  } else {
    if (lo) *reinterpret_cast<uint2*>(p) = make_uint2(r.v[0].x, r.v[0].y);
    if (hi) *reinterpret_cast<uint2*>(p + F) = make_uint2(r.v[0].z, r.v[0].w);
  }
}

// What stands for an absent gate, scale or shift: read like one, it keeps
// null checks out of the row loops (an absent gate or gain is 0 + 1).
__device__ __align__(16) float g_zeros[kMaxRowChannels];  // read as uint4

// Eight channels of a gate, scale, shift or weight; `step` between the fours.
SPARGE_DEV F8 load_mod(const float* m, int step) {
  Raw8<float> r;
  r.v[0] = __ldg(reinterpret_cast<const uint4*>(m));
  r.v[1] = __ldg(reinterpret_cast<const uint4*>(m + step));
  return f8(r);
}

// One such row as a thread sees it from row to row: in registers where it has
// them to spare; else in shared memory behind the ring (read through L1 instead,
// a third of it comes from L2: 583 instead of 476 us at 720p); where the ring
// leaves no room, through L1.
enum Where { kRegisters, kShared, kCached };
template <int V, Where WHERE>
struct Mod {
  const float* at;
  float plus;
  F8 kept;
  Ring ring;
  SPARGE_DEV void open(const float* row, float add_to, const int (&off)[V][2]) {
    at = row;
    plus = add_to;
    if constexpr (WHERE == kRegisters) {
      static_assert(V == 1, "eight channels");
      kept = add(load_mod(row + off[0][0], off[0][1]), f8(add_to));
    } else if constexpr (WHERE == kShared) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const F8 m = add(load_mod(row + off[v][0], off[v][1]), f8(add_to));
        reinterpret_cast<ulonglong2&>(ring[2 * v]) = make_ulonglong2(m.v[0], m.v[1]);
        reinterpret_cast<ulonglong2&>(ring[2 * v + 1]) = make_ulonglong2(m.v[2], m.v[3]);
      }
    }
  }
  SPARGE_DEV F8 get(int v, const int (&off)[V][2]) const {
    if constexpr (WHERE == kRegisters) {
      return kept;
    } else if constexpr (WHERE == kShared) {
      const ulonglong2 a = reinterpret_cast<const ulonglong2&>(ring[2 * v]);
      const ulonglong2 b = reinterpret_cast<const ulonglong2&>(ring[2 * v + 1]);
      return {{a.x, a.y, b.x, b.y}};
    } else {
      return add(load_mod(at + off[v][0], off[v][1]), f8(plus));
    }
  }
};
template <int V, Where WHERE>
constexpr int mod_pieces() {
  return WHERE == kShared ? 2 * V : 0;
}

// Mean and sum of squares about it of each of T rows over the slot.  `inv_cnt`: 1 /
// channels of this warp; `counts`: those of each warp of the slot.
template <int T, int V>
SPARGE_DEV void slot_moments(Slot& s, const F8 (&y)[T * V], const bool (&lo)[V],
                             const bool (&hi)[V], float inv_cnt, const float* counts, float inv_c,
                             float (&mean)[T], float (&m2)[T]) {
  float part[T];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    part[t] = total(y[t * V]);
#pragma unroll
    for (int v = 1; v < V; ++v) part[t] += total(y[t * V + v]);
  }
  const float mine = warp_sums(part, s.lane) * inv_cnt;
#pragma unroll
  for (int t = 0; t < T; ++t) {
    mean[t] = __shfl_sync(0xffffffffu, mine, t * (32 / T));
    part[t] = 0.f;
    const F8 m = f8(-mean[t]);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      F8 d = add(y[t * V + v], m);
      if (!lo[v]) d.v[0] = d.v[1] = 0;
      if (!hi[v]) d.v[2] = d.v[3] = 0;
      part[t] += dot(d, d);
    }
  }
  const float square = warp_sums(part, s.lane);
  if (s.W == 1) {
#pragma unroll
    for (int t = 0; t < T; ++t) m2[t] = __shfl_sync(0xffffffffu, square, t * (32 / T));
    return;
  }
  static_assert(2 * T <= kSlotRed, "reduction buffer");
  float* red = slot_half(s);
  if (s.lane % (32 / T) == 0)
    *reinterpret_cast<float2*>(red + s.warp * kSlotRed + 2 * (s.lane / (32 / T))) =
        make_float2(mine, square);
  slot_sync(s);
  // Lane l joins warps l % 8 (and l % 8 + 8) of row l / 8 % T.
  const int w = s.lane & 7;
  const float* in = red + w * kSlotRed + 2 * ((s.lane >> 3) % T);
  const float2 a = *reinterpret_cast<const float2*>(in);
  const float na = counts[w];
  float m, q;
  if constexpr (V == 1) {
    m = sum_of_8(na * a.x) * inv_c;
    const float da = a.x - m;
    q = sum_of_8(fmaf(na * da, da, a.y));
  } else {
    const float2 b = *reinterpret_cast<const float2*>(in + 8 * kSlotRed);
    const float nb = counts[w + 8];
    m = sum_of_8(fmaf(na, a.x, nb * b.x)) * inv_c;
    const float da = a.x - m, db = b.x - m;
    q = sum_of_8(fmaf(na * da, da, a.y) + fmaf(nb * db, db, b.y));
  }
#pragma unroll
  for (int t = 0; t < T; ++t) {
    mean[t] = __shfl_sync(0xffffffffu, m, 8 * t);
    m2[t] = __shfl_sync(0xffffffffu, q, 8 * t);
  }
}

// Rows a slot takes at once (backward with one: 144 instead of 140 us at 480p, 1017
// instead of 738 us at 720p in bf16), and pieces of one stage.
template <int V>
constexpr int fwd_rows() {
  return 2 / V;
}
template <int THREADS>
constexpr int bwd_rows() {
  return 2 / bwd_vectors(THREADS);
}
template <typename TX, typename TB, int V>
constexpr int fwd_pieces() {
  return fwd_rows<V>() * V * (pieces8<TX>() + pieces8<TB>());
}
template <typename TX, typename TB, int THREADS>
constexpr int bwd_pieces() {
  return bwd_rows<THREADS>() * bwd_vectors(THREADS) * 2 * (pieces8<TX>() + pieces8<TB>());
}
template <int V>
constexpr Where fwd_where() {
  return V == 1 ? kRegisters : kShared;
}
template <int THREADS>
constexpr Where bwd_where() {
  return THREADS == 192 ? kRegisters : THREADS == 640 ? kShared : kCached;
}
// CTAs of an SM that the forward's registers are budgeted for.  For wide rows the
// bound is left to the compiler: stated as one CTA it makes slower code (720p:
// 565 us against 487).
constexpr int fwd_residents(int V) { return V == 1 ? 3 : 2; }
// Stages of the ring; wide rows have as many as a CTA can hold.
template <typename TX, typename TB, int V>
constexpr int fwd_stages() {
  return V == 1 ? 2 : sizeof(TX) + sizeof(TB) == 8 ? 1 : 2;
}
template <typename TX, typename TB, int THREADS>
constexpr int bwd_stages() {
  constexpr int pieces = bwd_pieces<TX, TB, THREADS>();
  return THREADS == 192 ? 3 : THREADS == 640 ? (16 / pieces < 3 ? 16 / pieces : 3) : 24 / pieces;
}

// A thread's channels (vector v: fours at c + v * far and F further) and its
// part of the ring.
template <int V, int F, bool FULL>
struct Lane {
  int c, far;
  bool lo[V], hi[V], all;
  SPARGE_DEV bool low(int v) const { return FULL || lo[v]; }
  SPARGE_DEV bool high(int v) const { return FULL || hi[v]; }
  SPARGE_DEV bool full() const { return FULL || all; }
  int mod[V][2];  // where it reads a row that is kept: inside also behind the end
  Ring ring;
  SPARGE_DEV Lane(const Slot& s, int C, uint4* smem) {
    c = F == 4 ? s.tid * 8 : s.warp * 256 + s.lane * 4;
    far = s.W * 256;
    all = true;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      lo[v] = c + v * far < C;
      hi[v] = c + v * far + F < C;
      all = all && lo[v] && hi[v];
      mod[v][0] = lo[v] ? c + v * far : 0;
      mod[v][1] = hi[v] ? F : 0;
    }
    ring = {smem + threadIdx.x, static_cast<int>(blockDim.x)};
  }
};

// The rows of a slot's items.  An item is one of the `parts` interleaved
// shares of a group's rows: T rows of every parts * T, so that the slots of the
// machine read neighbouring rows at any time.
struct ItemWalk {
  int item, row, end, g;
  SPARGE_DEV void open(const ResnormParams& p, int T) {
    if (item >= p.items) return;
    g = item / p.parts;
    row = g * p.R + (item - g * p.parts) * T;
    end = (g + 1) * p.R;
  }
  SPARGE_DEV void next(const ResnormParams& p, int T, int nslots) {
    row += p.parts * T;
    if (row >= end) {
      item += nslots;
      open(p, T);
    }
  }
};

template <typename TX, typename TB, int V>
__global__ void __launch_bounds__(row_threads(V), V == 1 ? fwd_residents(V) : 0) resnorm_fwd_kernel(
    const __grid_constant__ ResnormParams p) {
  constexpr int T = fwd_rows<V>(), S = fwd_stages<TX, TB, V>(), XQ = pieces8<TX>(), BQ = pieces8<TB>();
  constexpr int PIECES = fwd_pieces<TX, TB, V>(), STAGE = PIECES;
  extern __shared__ uint4 smem[];
  __shared__ __align__(16) float red[red_floats(row_threads(V))];
  __shared__ float counts[16];  // a slot of the forward has at most 16 warps
  Slot s = make_slot(p.W, red, red_half(row_threads(V)));
  const int per_cta = slots_per_cta(p.W);
  if (threadIdx.x < 16) {
    // Channels of each warp of a slot, none of those it does not have.
    int n = 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (threadIdx.x < p.W)
        n += max(0, min(256, p.C - (v * p.W + static_cast<int>(threadIdx.x)) * 256));
    counts[threadIdx.x] = static_cast<float>(n);
  }
  __syncthreads();
  if (s.index >= per_cta) return;
  const float inv_cnt = 1.f / counts[s.warp];
  constexpr int F = four_step<TX>();
  const Lane<V, F, false> at(s, p.C, smem);
  // What is never loaded is zero: threads behind the last channel add zeros.
  if (!at.all) {
    for (int k = 0; k < S * PIECES; ++k) at.ring[k] = make_uint4(0, 0, 0, 0);
  }

  const int nslots = static_cast<int>(gridDim.x) * per_cta;
  ItemWalk ahead = {static_cast<int>(blockIdx.x) * per_cta + s.index, 0, 0, 0};
  ahead.open(p, T);
  ItemWalk now = ahead;

  const TX* x = static_cast<const TX*>(p.x) + at.c;
  const TB* b = static_cast<const TB*>(p.b) + at.c;
  const bool has_b = p.b != nullptr, has_post = p.post != nullptr;
  const auto issue = [&](Ring stage) {
    if (ahead.item < p.items) {
      int64_t o = static_cast<int64_t>(ahead.row) * p.C;
#pragma unroll
      for (int t = 0; t < T; ++t) {
        if (ahead.row + t < ahead.end) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const Ring dst = stage + (t * V + v) * (XQ + BQ);
            stage_fours<F>(dst, x + o + v * at.far, at.lo[v], at.hi[v]);
            if (has_b) stage_fours<F>(dst + XQ, b + o + v * at.far, at.lo[v], at.hi[v]);
          }
        }
        o += p.C;
      }
      ahead.next(p, T, nslots);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < S; ++k) issue(at.ring + k * STAGE);

  const float* gate_row = (p.gate != nullptr ? p.gate : g_zeros);
  const float* scale_row = (p.scale != nullptr ? p.scale : g_zeros);
  const float* shift_row = (p.shift != nullptr ? p.shift : g_zeros);
  const float plus = p.unit || p.scale == nullptr ? 1.f : 0.f;
  const float gate_plus = p.gate == nullptr ? 1.f : 0.f;
  constexpr Where WHERE = fwd_where<V>();
  constexpr int KEPT = mod_pieces<V, WHERE>();
  Mod<V, WHERE> gate, gain, shift;
  gate.ring = at.ring + S * PIECES;
  gain.ring = gate.ring + KEPT;
  shift.ring = gain.ring + KEPT;
  int group = -1;
  int k = 0;
  while (now.item < p.items) {
    const int rows = min(T, now.end - now.row), row = now.row;
    if (now.g != group) {
      group = now.g;
      gate.open(gate_row + group * p.gate_ld, gate_plus, at.mod);
      gain.open(scale_row + group * p.scale_ld, plus, at.mod);
      shift.open(shift_row + group * p.shift_ld, 0.f, at.mod);
    }
    now.next(p, T, nslots);
    // The stage is read out at once and filled again, so its bytes are in
    // flight while the rows are computed.
    cp_async_wait<S - 1>();
    const Ring stage = at.ring + k * STAGE;
    k = k + 1 == S ? 0 : k + 1;
    Raw8<TX> rx[T * V];
    Raw8<TB> rb[T * V];
#pragma unroll
    for (int i = 0; i < T * V; ++i) {
      rx[i] = unstage8<TX>(stage + i * (XQ + BQ));
      rb[i] = unstage8<TB>(stage + i * (XQ + BQ) + XQ);
    }
    issue(stage);
    F8 y[T * V];
    float rbs[T];
    if (has_b) {
      F8 b8[T * V];
#pragma unroll
      for (int i = 0; i < T * V; ++i) b8[i] = f8(rb[i]);
      if (has_post) {
#pragma unroll
        for (int t = 0; t < T; ++t) {
          rbs[t] = dot(b8[t * V], b8[t * V]);
#pragma unroll
          for (int v = 1; v < V; ++v) rbs[t] += dot(b8[t * V + v], b8[t * V + v]);
        }
        slot_sum<warp_eights(row_threads(V))>(s, rbs);
#pragma unroll
        for (int t = 0; t < T; ++t) {
          rbs[t] = rsqrtf(rbs[t] * p.inv_c + p.eps);
#pragma unroll
          for (int v = 0; v < V; ++v)
            b8[t * V + v] = mul(mul(b8[t * V + v], f8(rbs[t])),
                                load_mod(p.post + at.mod[v][0], at.mod[v][1]));
        }
      }
      int64_t o = static_cast<int64_t>(row) * p.C + at.c;
#pragma unroll
      for (int t = 0; t < T; ++t) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int i = t * V + v;
          y[i] = fma(gate.get(v, at.mod), b8[i], f8(rx[i]));
          if (t < rows) put<F>(static_cast<TX*>(p.y) + o + v * at.far, y[i], at.lo[v], at.hi[v]);
        }
        o += p.C;
      }
    } else {
#pragma unroll
      for (int i = 0; i < T * V; ++i) y[i] = f8(rx[i]);
    }
    float mean[T], rstd[T];
    if (p.norm != SPARGE_NORM_NONE) {
      if (p.norm == SPARGE_NORM_LAYER) {
        slot_moments<T, V>(s, y, at.lo, at.hi, inv_cnt, counts, p.inv_c, mean, rstd);
      } else {
#pragma unroll
        for (int t = 0; t < T; ++t) {
          mean[t] = 0.f;
          rstd[t] = dot(y[t * V], y[t * V]);
#pragma unroll
          for (int v = 1; v < V; ++v) rstd[t] += dot(y[t * V + v], y[t * V + v]);
        }
        slot_sum<warp_eights(row_threads(V))>(s, rstd);
      }
      int64_t o = static_cast<int64_t>(row) * p.C + at.c;
#pragma unroll
      for (int t = 0; t < T; ++t) {
        rstd[t] = rsqrtf(rstd[t] * p.inv_c + p.eps);
        const F8 m = f8(-mean[t]), r = f8(rstd[t]);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const F8 h = fma(mul(add(y[t * V + v], m), r), gain.get(v, at.mod), shift.get(v, at.mod));
          if (t < rows) put<F>(static_cast<TB*>(p.h) + o + v * at.far, h, at.lo[v], at.hi[v]);
        }
        o += p.C;
      }
    }
    if (s.tid == 0 && p.stats != nullptr) {
#pragma unroll
      for (int t = 0; t < T; ++t) {
        if (t >= rows) continue;
        if (p.norm != SPARGE_NORM_NONE) {
          p.stats[row + t] = mean[t];
          p.stats[p.M + row + t] = rstd[t];
        }
        if (has_post) p.stats[2 * static_cast<int64_t>(p.M) + row + t] = rbs[t];
      }
    }
  }
}

// FULL: every input is there and no thread is without channels, which takes the
// branches out of the row loop (one modulation a frame, both norms, 480p: 124
// instead of 155 us).
template <typename TX, typename TB, int THREADS, bool POST, bool FULL>
__global__ void __launch_bounds__(THREADS, THREADS == 192 ? 2 : 0) resnorm_bwd_kernel(
    const __grid_constant__ ResnormParams p) {
  constexpr int V = bwd_vectors(THREADS), T = bwd_rows<THREADS>(),
                S = bwd_stages<TX, TB, THREADS>(), XQ = pieces8<TX>(), BQ = pieces8<TB>();
  constexpr int PIECES = bwd_pieces<TX, TB, THREADS>(), ROW = 2 * (XQ + BQ), STAGE = PIECES;
  constexpr int SUMS = POST ? 4 : 3;
  extern __shared__ uint4 smem[];
  __shared__ __align__(16) float red[red_floats(THREADS)];
  grid_launch_dependents();
  Slot s = make_slot(p.W, red, red_half(THREADS));
  __syncthreads();
  const int per_cta = slots_per_cta(p.W);
  if (s.index >= per_cta) return;
  constexpr int F = four_step<TX>();
  const Lane<V, F, FULL> at(s, p.C, smem);
  const bool normed = FULL || p.norm != SPARGE_NORM_NONE, has_b = FULL || p.b != nullptr;
  const bool has_dy = FULL || p.dy != nullptr, has_dh = FULL || p.dh != nullptr;
  F8 acc[SUMS][V];  // gate, scale, shift, post
#pragma unroll
  for (int k = 0; k < SUMS; ++k) {
#pragma unroll
    for (int v = 0; v < V; ++v) acc[k][v] = f8(0.f);
  }
  // What is never loaded is zero: absent inputs, threads behind the last channel.
  if (!(at.full() && normed && has_b && has_dy && has_dh)) {
    for (int k = 0; k < S * PIECES; ++k) at.ring[k] = make_uint4(0, 0, 0, 0);
  }

  const int nslots = gridDim.x * per_cta, slot = blockIdx.x * per_cta + s.index;
  ItemWalk ahead = {slot, 0, 0, 0};
  ahead.open(p, T);
  ItemWalk now = ahead;
  const TX* x = static_cast<const TX*>(p.x) + at.c;
  const TB* b = static_cast<const TB*>(p.b) + at.c;
  const TX* dy = static_cast<const TX*>(p.dy) + at.c;
  const TB* dh = static_cast<const TB*>(p.dh) + at.c;
  const auto issue = [&](Ring stage) {
    if (ahead.item < p.items) {
      int64_t o = static_cast<int64_t>(ahead.row) * p.C;
#pragma unroll
      for (int t = 0; t < T; ++t) {
        if (ahead.row + t < ahead.end) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const Ring dst = stage + (t * V + v) * ROW;
            const int64_t ov = o + v * at.far;
            if (normed) stage_fours<F>(dst, x + ov, at.low(v), at.high(v));
            if (has_b) stage_fours<F>(dst + XQ, b + ov, at.low(v), at.high(v));
            if (has_dy) stage_fours<F>(dst + XQ + BQ, dy + ov, at.low(v), at.high(v));
            if (has_dh) stage_fours<F>(dst + 2 * XQ + BQ, dh + ov, at.low(v), at.high(v));
          }
        }
        o += p.C;
      }
      ahead.next(p, T, nslots);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < S; ++k) issue(at.ring + k * STAGE);

  // The row's mean, 1/deviation and branch 1/rms, one step ahead.
  float mean_n[T], rstd_n[T], rb_n[T];
  const auto fetch = [&](const ItemWalk& w) {
#pragma unroll
    for (int t = 0; t < T; ++t) {
      mean_n[t] = rstd_n[t] = 0.f;
      rb_n[t] = 1.f;
      if (w.item < p.items && w.row + t < w.end) {
        if (p.norm == SPARGE_NORM_LAYER) mean_n[t] = p.stats[w.row + t];
        if (normed) rstd_n[t] = p.stats[p.M + w.row + t];
        if (POST) rb_n[t] = p.stats[2 * static_cast<int64_t>(p.M) + w.row + t];
      }
    }
  };
  fetch(now);

  const float* gate_row = (p.gate != nullptr ? p.gate : g_zeros);
  const float* scale_row = (p.scale != nullptr ? p.scale : g_zeros);
  const float plus = p.unit || p.scale == nullptr ? 1.f : 0.f;
  const float gate_plus = p.gate == nullptr ? 1.f : 0.f;
  const float one_mean = p.norm == SPARGE_NORM_LAYER ? p.inv_c : 0.f;
  constexpr Where WHERE = bwd_where<THREADS>();
  constexpr int KEPT = mod_pieces<V, WHERE>();
  Mod<V, WHERE> gate, gain, post;
  gate.ring = at.ring + S * PIECES;
  gain.ring = gate.ring + KEPT;
  post.ring = gain.ring + KEPT;
  if (POST) post.open(p.post, 0.f, at.mod);
  int group = -1;
  int k = 0;
  while (now.item < p.items) {
    const int item = now.item, rows = min(T, now.end - now.row), row = now.row;
    if (now.g != group) {
      group = now.g;
      gate.open(gate_row + group * p.gate_ld, gate_plus, at.mod);
      gain.open(scale_row + group * p.scale_ld, plus, at.mod);
    }
    float mean[T], rstd[T], rb[T];
#pragma unroll
    for (int t = 0; t < T; ++t) mean[t] = mean_n[t], rstd[t] = rstd_n[t], rb[t] = rb_n[t];
    now.next(p, T, nslots);
    fetch(now);
    cp_async_wait<S - 1>();
    const Ring stage = at.ring + k * STAGE;
    k = k + 1 == S ? 0 : k + 1;

    F8 z[T * V], d[T * V];
    float sums[2 * T] = {};
    if (normed) {
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const F8 m = f8(-mean[t]), r = f8(rstd[t]);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int i = t * V + v;
          const Ring src = stage + i * ROW;
          F8 y = unstage<TX>(src);
          if (has_b) {
            F8 n = unstage<TB>(src + XQ);
            if (POST) n = mul(mul(n, f8(rb[t])), post.get(v, at.mod));
            y = fma(gate.get(v, at.mod), n, y);
          }
          z[i] = mul(add(y, m), r);
          const F8 h = unstage<TB>(src + 2 * XQ + BQ);
          d[i] = mul(h, gain.get(v, at.mod));
          if (t < rows) {
            acc[1][v] = fma(h, z[i], acc[1][v]);
            acc[2][v] = add(acc[2][v], h);
          }
          sums[2 * t] += total(d[i]);
          sums[2 * t + 1] += dot(d[i], z[i]);
        }
      }
      slot_sum<warp_eights(THREADS)>(s, sums);
    }
    float e[T];
    int64_t o = static_cast<int64_t>(row) * p.C + at.c;
#pragma unroll
    for (int t = 0; t < T; ++t) {
      e[t] = 0.f;
      if (t < rows) {
        const F8 c1 = f8(-sums[2 * t] * one_mean), c2 = f8(-sums[2 * t + 1] * p.inv_c);
        const F8 r = f8(rstd[t]);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int i = t * V + v;
          const Ring src = stage + i * ROW;
          const F8 g = unstage<TX>(src + XQ + BQ);
          d[i] = normed ? fma(r, fma(z[i], c2, add(d[i], c1)), g) : g;
          put<F>(static_cast<TX*>(p.dx) + o + v * at.far, d[i], at.low(v), at.high(v));
          if (!has_b) continue;
          const F8 b8 = unstage<TB>(src + XQ);
          if (POST) {
            const F8 bh = mul(b8, f8(rb[t])), w = post.get(v, at.mod);
            acc[0][v] = fma(d[i], mul(bh, w), acc[0][v]);
            d[i] = mul(d[i], gate.get(v, at.mod));
            acc[SUMS - 1][v] = fma(d[i], bh, acc[SUMS - 1][v]);
            d[i] = mul(d[i], w);
            e[t] += dot(d[i], bh);  // bh is 0 behind the last channel
          } else {
            acc[0][v] = fma(d[i], b8, acc[0][v]);
            d[i] = mul(d[i], gate.get(v, at.mod));
            put<F>(static_cast<TB*>(p.db) + o + v * at.far, d[i], at.low(v), at.high(v));
          }
        }
      }
      o += p.C;
    }
    if (POST) {
      slot_sum<warp_eights(THREADS)>(s, e);
      o = static_cast<int64_t>(row) * p.C + at.c;
#pragma unroll
      for (int t = 0; t < T; ++t) {
        if (t < rows) {
          const F8 r = f8(rb[t]), c3 = f8(-e[t] * p.inv_c * rb[t]);
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const int i = t * V + v;
            const F8 b8 = unstage<TB>(stage + i * ROW + XQ);
            put<F>(static_cast<TB*>(p.db) + o + v * at.far, mul(fma(b8, c3, d[i]), r), at.low(v),
                   at.high(v));
          }
        }
        o += p.C;
      }
    }
    issue(stage);

    if (now.item != item) {  // the item's last rows
#pragma unroll
      for (int j = 0; j < SUMS; ++j) {
        if (!p.by_group[j]) continue;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (p.sum[j] != nullptr)
            put<F>(p.sum[j] + static_cast<int64_t>(item) * p.C + at.c + v * at.far, acc[j][v],
                   at.low(v), at.high(v));
          acc[j][v] = f8(0.f);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < SUMS; ++j) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!p.by_group[j] && p.sum[j] != nullptr)
        put<F>(p.sum[j] + static_cast<int64_t>(slot) * p.C + at.c + v * at.far, acc[j][v],
               at.low(v), at.high(v));
    }
  }
}

struct ResnormPlan {
  int V, W, per_cta, threads, ctas, slots, smem;
  int built;  // the size of CTA that the backward kernel is built for
  int groups, R;
  int items, parts;  // items = groups * parts
  // backward: a sum is written per item straight to the output (one part a
  // group), per item to the workspace, or per slot to the workspace
  bool wanted[4], by_group[4];
  size_t off[4], bytes;
};

template <typename TX, typename TB, int V>
constexpr int fwd_ring() {
  return fwd_stages<TX, TB, V>() * fwd_pieces<TX, TB, V>() + 3 * mod_pieces<V, fwd_where<V>()>();
}
template <typename TX, typename TB, int THREADS>
constexpr int bwd_ring() {
  return bwd_stages<TX, TB, THREADS>() * bwd_pieces<TX, TB, THREADS>() +
         3 * mod_pieces<bwd_vectors(THREADS), bwd_where<THREADS>()>();
}
// Pieces of a thread's ring, with the rows that it keeps.
template <typename TX, typename TB>
int ring_pieces(int V, int threads, bool bwd) {
  if (!bwd) return V == 1 ? fwd_ring<TX, TB, 1>() : fwd_ring<TX, TB, 2>();
  return threads == 192   ? bwd_ring<TX, TB, 192>()
         : threads == 640 ? bwd_ring<TX, TB, 640>()
                          : bwd_ring<TX, TB, 512>();
}

constexpr int kDeclared = 4672;  // shared memory that a kernel declares, at most

ResnormPlan resnorm_plan(const sparge_resnorm& a, bool bwd) {
  ResnormPlan pl = {};
  const int64_t M = a.rows;
  pl.built = bwd ? bwd_threads(a.C) : 0;
  pl.V = bwd ? bwd_vectors(pl.built) : row_vectors(a.C);
  pl.W = slot_warps(a.C, pl.V);
  pl.per_cta = slots_per_cta(pl.W);
  pl.threads = pl.W * pl.per_cta * 32;
  const int ring =
      a.x_type == SPARGE_BF16 ? ring_pieces<__nv_bfloat16, __nv_bfloat16>(pl.V, pl.built, bwd)
      : a.branch_type == SPARGE_BF16 ? ring_pieces<float, __nv_bfloat16>(pl.V, pl.built, bwd)
                                     : ring_pieces<float, float>(pl.V, pl.built, bwd);
  pl.smem = ring * pl.threads * 16;
  int groups = 1;
  if (a.gate) groups = std::max(groups, a.gate_groups);
  if (a.scale) groups = std::max(groups, a.scale_groups);
  if (a.shift) groups = std::max(groups, a.shift_groups);
  pl.groups = groups;
  pl.R = static_cast<int>(M / groups);
  const int T = 2 / pl.V;
  // CTAs that are resident at a time: shared memory limits them, or registers.
  // The backward stays resident for its share of the rows, since every slot
  // leaves a row of sums; the forward runs several waves, whose CTAs end one by
  // one instead of all at once with the slowest (480p: one wave 104 us, two 101,
  // eight 93; 720p: four).
  const int warps = pl.threads / 32;
  const int by_regs = bwd ? resident_warps(bwd_regs(pl.built)) / warps
                          : fwd_residents(pl.V) * row_threads(pl.V) / pl.threads;
  const int per_sm = std::max(1, std::min(std::min(by_regs, 64 / warps),
                                          kSmemPerSm / (pl.smem + kSmemOfCta + kDeclared)));
  const int waves = bwd ? 1 : pl.V == 1 ? 8 : 4;
  const int64_t most = static_cast<int64_t>(kSMs) * per_sm * waves;
  const int64_t target = most * pl.per_cta;  // slots that fill the machine
  const int64_t units = (pl.R + T - 1) / T;
  pl.parts = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(units, target / groups)));
  pl.items = groups * pl.parts;
  pl.ctas = static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>(most, (static_cast<int64_t>(pl.items) + pl.per_cta - 1) / pl.per_cta)));
  pl.slots = pl.ctas * pl.per_cta;
  if (!bwd) return pl;
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
  return p;
}

template <int PIECES, int THREADS, typename Kernel>
cudaError_t launch_kernel(Kernel* kernel, const ResnormParams& p, const ResnormPlan& pl,
                          cudaStream_t st) {
  constexpr int most = 16 * PIECES * THREADS;  // the rings of all the threads it is built for
  static_assert(most + kDeclared <= kSmemPerCta, "shared memory of a CTA");
  return launch_row_kernel(kernel, p, dim3(pl.ctas), pl.threads, pl.smem, most, st);
}

template <typename TX, typename TB, int V>
cudaError_t launch_fwd(const ResnormParams& p, const ResnormPlan& pl, cudaStream_t st) {
  return launch_kernel<fwd_ring<TX, TB, V>(), row_threads(V)>(resnorm_fwd_kernel<TX, TB, V>, p, pl,
                                                              st);
}

template <typename TX, typename TB, int THREADS>
cudaError_t launch_bwd(const ResnormParams& p, const ResnormPlan& pl, cudaStream_t st) {
  // (Sixteen channels a thread leave no registers for the full form.)
  constexpr bool kFull = bwd_vectors(THREADS) == 1;
  const bool post = p.post != nullptr;
  const bool full = kFull && p.C % 256 == 0 && p.norm && p.b && p.dy && p.dh;
  auto* kernel = full ? (post ? resnorm_bwd_kernel<TX, TB, THREADS, true, kFull>
                              : resnorm_bwd_kernel<TX, TB, THREADS, false, kFull>)
                      : (post ? resnorm_bwd_kernel<TX, TB, THREADS, true, false>
                              : resnorm_bwd_kernel<TX, TB, THREADS, false, false>);
  return launch_kernel<bwd_ring<TX, TB, THREADS>(), THREADS>(kernel, p, pl, st);
}

template <typename TX, typename TB>
cudaError_t launch_resnorm(const ResnormParams& p, const ResnormPlan& pl, bool bwd,
                           cudaStream_t st) {
  if (bwd) {
    if (pl.built == 192) return launch_bwd<TX, TB, 192>(p, pl, st);
    if (pl.built == 640) return launch_bwd<TX, TB, 640>(p, pl, st);
    return launch_bwd<TX, TB, 512>(p, pl, st);
  }
  return pl.V == 1 ? launch_fwd<TX, TB, 1>(p, pl, st) : launch_fwd<TX, TB, 2>(p, pl, st);
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
