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
//
// Bound by memory: forward reads and writes every value once, backward reads the
// gradient and the input and writes once (no normed row is kept for it; r comes
// from the input again).  A row's statistics need all of its channels, so a slot
// of warps holds a whole token and both tensors share its angles, computed once
// for all heads.  Measured, bf16, norm over the token: 32760 tokens of 12 x 128,
// Q, K and V: forward 96 us for 604 MB (6.3 TB/s), backward 129 us for 805 MB
// (6.2 TB/s); 75600 tokens of 40 x 128: 780 us for 4.64 GB (5.9 TB/s) and 1075
// us for 6.2 GB (5.8 TB/s).  What is missing to a copy's 6.8 TB/s is latency: 12
// warps an SM (20 in the wide backward), and a barrier a unit.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "common.cuh"
#include "places.h"
#include "rows.cuh"
#include "sparge.h"

namespace sparge {

namespace {

struct HeadsPart {
  const void* x;
  const void* w;
  void* y;  // head-major bf16: the result, or the gradient that comes back
  void* dx;
  float* dw_part;  // [CTAs][H * d] or, under a norm over each head, [CTAs][d]
  int64_t xs[3], ds[3];
  // From a slot's unit to its next: samples and tokens, the same in elements of
  // x, y and dx, and what to add where the token would lie behind the sample.
  int db, dn;
  int64_t x_step, y_step, d_step, x_wrap, y_wrap, d_wrap;
  int C, W, plain;
  SPARGE_DEV void advance(int span, int& b, int& n) const {
    b += db;
    n += dn;
    if (n >= span) n -= span, ++b;
  }
};
// The element of a part at which a thread's channels of a token begin.
SPARGE_DEV int64_t part_at(const int64_t (&stride)[3], int b, int n, int head, int c) {
  return b * stride[0] + n * stride[1] + head * stride[2] + c;
}

struct HeadsParams {
  HeadsPart part[3];
  const int32_t* grid;
  const int32_t* pos;
  int64_t pos_ld;  // elements between samples of pos
  int M, N;        // rows in all, rows of one sample
  int span;        // N rounded up to whole units
  int norm, rotate, w_bf16;
  float eps;
  uint64_t turn[64];
  uint8_t axis[64];
};

// Frequencies in shared memory: indexed by lane, they would be replayed 32
// times out of the parameter bank.
struct Turns {
  uint64_t turn[64];
  uint8_t axis[64];
  SPARGE_DEV void fill(const HeadsParams& p) {
    if (threadIdx.x < 64) {
      turn[threadIdx.x] = p.turn[threadIdx.x];
      axis[threadIdx.x] = p.axis[threadIdx.x];
    }
  }
};

// The cosines and sines of a slot's tokens, T at a time, each computed once for
// all heads of its parts: [T][cos | sin][D / 2] floats of shared memory.
// Thread i of the slot owns pair i % (D / 2) of token i / (D / 2) (and more of
// them where the slot is narrow).  Coordinates are counted on from unit to
// unit, so the divisions are done once a sample.
template <int T, int D>
struct Angles {
  static constexpr int P = D / 2;
  int n, b;        // the next token
  int it, ih, iw;  // its coordinates on the grid
  int t, h, w;     // the sample's grid; t = 0: nothing turns
  int dt, dh, dw;  // a step between units, as coordinates
  int held;        // a given position (of the thread's first pair), read a unit
                   // ahead: read when it is needed, 480p takes 122 us, not 97

  SPARGE_DEV void open(const HeadsParams& p, int sample, int token, int dn) {
    b = sample;
    n = token;
    it = ih = iw = t = 0;
    if (p.grid == nullptr || b * static_cast<int64_t>(p.N) >= p.M) return;
    const int32_t* size = p.grid + 3 * static_cast<int64_t>(b);  // (past 2^31 with N = 1)
    t = size[0], h = size[1], w = size[2];
    if (t < 1 || h < 1 || w < 1) {
      t = 0;
      return;
    }
    place(n, it, ih, iw);
    place(dn, dt, dh, dw);
  }
  SPARGE_DEV void place(int token, int& ct, int& ch, int& cw) const {
    const int64_t hw = static_cast<int64_t>(h) * w;
    ct = hw > token ? 0 : token / static_cast<int>(hw);
    const int rest = token - static_cast<int>(ct * hw);
    ch = rest / w;
    cw = rest - ch * w;
  }
  // The position of the token `on` (0 or 1) tokens on along axis a.
  SPARGE_DEV int position(const HeadsParams& p, int on, int a) const {
    if (p.pos != nullptr)
      return n + on < p.N && b * static_cast<int64_t>(p.N) < p.M
                 ? p.pos[b * p.pos_ld + static_cast<int64_t>(n + on) * 3 + a]
                 : 0;
    int ct = it, ch = ih, cw = iw;
    if (T > 1 && on != 0) step(ct, ch, cw);
    if (ct >= t) return 0;  // behind the grid, or no grid
    return a == 0 ? ct : a == 1 ? ch : cw;
  }
  SPARGE_DEV void step(int& ct, int& ch, int& cw) const {
    if (++cw == w) {
      cw = 0;
      if (++ch == h) ch = 0, ++ct;
    }
  }
  SPARGE_DEV void hold(const HeadsParams& p, const Slot& s, const Turns& turns) {
    if (p.pos != nullptr && s.tid < T * P) held = position(p, s.tid / P, turns.axis[s.tid % P]);
  }
  SPARGE_DEV void fill(const HeadsParams& p, const Slot& s, const Turns& turns, float* out) {
    for (int i = s.tid; i < T * P; i += s.W * 32) {
      const int j = i % P;
      const int pos =
          p.pos != nullptr && i == s.tid ? held : position(p, i / P, turns.axis[j]);
      const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * turns.turn[j];
      float c, q;
      sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f, &q,
                &c);  // 2^-31: half turns
      out[(i / P) * D + j] = c;
      out[(i / P) * D + P + j] = q;
    }
  }
  // On to the slot's next unit.
  SPARGE_DEV void next(const HeadsParams& p, const HeadsPart& part, const Slot& s,
                       const Turns& turns) {
    const int before = b;
    part.advance(p.span, b, n);
    if (b != before) {
      open(p, b, n, part.dn);
    } else if (t > 0) {
      iw += dw;
      ih += dh;
      it += dt;
      if (iw >= w) iw -= w, ++ih;
      if (ih >= h) ih -= h, ++it;
    }
    hold(p, s, turns);
  }
  SPARGE_DEV void start(const HeadsParams& p, const HeadsPart& part, const Slot& s,
                        const Turns& turns, int sample, int token) {
    open(p, sample, token, part.dn);
    hold(p, s, turns);
  }
};

// Four pairs (a, b) of a thread as packed halves: a[0] holds the first members
// of pairs 0 and 1.  Both channel orders unpack into it and pack out of it
// without a move, and every step below is a packed operation.
struct Pairs {
  uint64_t a[2], b[2];
};

template <bool INTER>
SPARGE_DEV Pairs to_pairs(const float (&f)[8]) {
  if constexpr (INTER)
    return {{f32x2(f[0], f[2]), f32x2(f[4], f[6])}, {f32x2(f[1], f[3]), f32x2(f[5], f[7])}};
  else
    return {{f32x2(f[0], f[1]), f32x2(f[2], f[3])}, {f32x2(f[4], f[5]), f32x2(f[6], f[7])}};
}
template <bool INTER>
SPARGE_DEV void from_pairs(const Pairs& v, float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float a = j & 1 ? f32x2_hi(v.a[j / 2]) : f32x2_lo(v.a[j / 2]);
    const float b = j & 1 ? f32x2_hi(v.b[j / 2]) : f32x2_lo(v.b[j / 2]);
    f[INTER ? 2 * j : j] = a;
    f[INTER ? 2 * j + 1 : j + 4] = b;
  }
}

SPARGE_DEV float dot(const Pairs& x, const Pairs& y) {
  const uint64_t s = ffma2(x.a[0], y.a[0], fmul2(x.b[0], y.b[0]));
  const uint64_t t = ffma2(x.a[1], y.a[1], fmul2(x.b[1], y.b[1]));
  const uint64_t u = fadd2(s, t);
  return f32x2_lo(u) + f32x2_hi(u);
}
SPARGE_DEV Pairs mul(const Pairs& x, const Pairs& y) {
  return {{fmul2(x.a[0], y.a[0]), fmul2(x.a[1], y.a[1])},
          {fmul2(x.b[0], y.b[0]), fmul2(x.b[1], y.b[1])}};
}
SPARGE_DEV Pairs mul(const Pairs& x, float f) {
  const uint64_t r = f32x2(f, f);
  return {{fmul2(x.a[0], r), fmul2(x.a[1], r)}, {fmul2(x.b[0], r), fmul2(x.b[1], r)}};
}
SPARGE_DEV Pairs fma(const Pairs& x, const Pairs& y, const Pairs& z) {
  return {{ffma2(x.a[0], y.a[0], z.a[0]), ffma2(x.a[1], y.a[1], z.a[1])},
          {ffma2(x.b[0], y.b[0], z.b[0]), ffma2(x.b[1], y.b[1], z.b[1])}};
}
SPARGE_DEV Pairs fma(const Pairs& x, float f, const Pairs& z) {
  const uint64_t r = f32x2(f, f);
  return {{ffma2(x.a[0], r, z.a[0]), ffma2(x.a[1], r, z.a[1])},
          {ffma2(x.b[0], r, z.b[0]), ffma2(x.b[1], r, z.b[1])}};
}

// A thread's four angles of a token: pairs c / 2 on where its channels are eight
// in a row from c, pairs c on where they are partners, else c / 2 and c / 2 + 1
// and the same a quarter of a head on.
template <bool INTER, bool SPLIT, int D>
SPARGE_DEV float4 four_of(const float* row, int c) {
  if constexpr (!SPLIT) {
    return *reinterpret_cast<const float4*>(row + c / 2);
  } else if constexpr (!INTER) {
    return *reinterpret_cast<const float4*>(row + c);
  } else {
    const float2 a = *reinterpret_cast<const float2*>(row + c / 2);
    const float2 b = *reinterpret_cast<const float2*>(row + c / 2 + D / 4);
    return make_float4(a.x, a.y, b.x, b.y);
  }
}

// Turns the pairs by the angles at cs (BACK: by their negatives).
template <bool BACK, bool INTER, bool SPLIT, int D>
SPARGE_DEV Pairs rotate(const Pairs& v, const float* cs, int at) {
  const float4 c4 = four_of<INTER, SPLIT, D>(cs, at);
  const float4 s4 = four_of<INTER, SPLIT, D>(cs + D / 2, at);
  const uint64_t c[2] = {f32x2(c4.x, c4.y), f32x2(c4.z, c4.w)};
  const uint64_t s[2] = {f32x2(s4.x, s4.y), f32x2(s4.z, s4.w)};
  const uint64_t n[2] = {f32x2(-s4.x, -s4.y), f32x2(-s4.z, -s4.w)};
  Pairs r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    r.a[i] = ffma2(v.a[i], c[i], fmul2(v.b[i], BACK ? s[i] : n[i]));
    r.b[i] = ffma2(v.a[i], BACK ? n[i] : s[i], fmul2(v.b[i], c[i]));
  }
  return r;
}

// A thread's eight channels of one token: eight in a row for bf16 with adjacent
// pairs, else four and the four that lie half a head further: their partners,
// or two more pairs, so that fp32 rows too are read in whole sectors.
template <typename TX, bool INTER>
constexpr bool split() {
  return !INTER || sizeof(TX) == 4;
}
template <typename T, bool SPLIT, int D>
SPARGE_DEV void stage_row(Ring dst, const T* p) {
  if constexpr (!SPLIT)
    stage8(dst, p);
  else
    stage4x2(dst, p, p + D / 2);
}
template <bool SPLIT, int D>
SPARGE_DEV void store_row_raw(__nv_bfloat16* p, const Raw8<__nv_bfloat16>& r) {
  if constexpr (!SPLIT) {
    store_raw8(p, r);
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(r.v[0].x, r.v[0].y);
    *reinterpret_cast<uint2*>(p + D / 2) = make_uint2(r.v[0].z, r.v[0].w);
  }
}
template <typename T, bool SPLIT, int D>
SPARGE_DEV void store_row(T* p, const float (&f)[8]) {
  if constexpr (!SPLIT)
    store8(p, f);
  else
    store4x2(p, p + D / 2, f);
}
template <typename T, bool INTER>
SPARGE_DEV Pairs unstage_pairs(Ring src) {
  float f[8];
  unpack8(unstage8<T>(src), f);
  return to_pairs<INTER>(f);
}
// The weights lie in the ring in the order of the pairs.
SPARGE_DEV Pairs unstage_weight(Ring src) {
  const ulonglong2 a = reinterpret_cast<const ulonglong2&>(src[0]);
  const ulonglong2 b = reinterpret_cast<const ulonglong2&>(src[1]);
  return {{a.x, a.y}, {b.x, b.y}};
}
SPARGE_DEV void keep_weight(Ring dst, const Pairs& w) {
  reinterpret_cast<ulonglong2&>(dst[0]) = make_ulonglong2(w.a[0], w.a[1]);
  reinterpret_cast<ulonglong2&>(dst[1]) = make_ulonglong2(w.b[0], w.b[1]);
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

// The weights of this thread's eight channels (1 without a weight).
template <bool INTER, bool SPLIT, int D>
SPARGE_DEV Pairs load_weight(const HeadsParams& p, const void* w, bool active, int c) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = c + (!SPLIT || i < 4 ? i : i - 4 + D / 2);
    f[i] = 1.f;
    if (w != nullptr && active)
      f[i] = p.w_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[at])
                      : static_cast<const float*>(w)[at];
  }
  return to_pairs<INTER>(f);
}

// A thread's place in the rows of a part: vector v of V covers eight channels
// of head `head + v * head_step`, from channel c of the head.
template <bool SPLIT, int D, int V, bool FULL>
struct Place {
  bool active[V];
  int head, head_step, c;
  SPARGE_DEV bool here(int v) const { return FULL || active[v]; }
  SPARGE_DEV Place(const Slot& s, int C) {
    constexpr int L = D / 8;  // threads of one head
#pragma unroll
    for (int v = 0; v < V; ++v) active[v] = (s.tid + v * s.W * 32) * 8 < C;
    head = s.tid / L;
    head_step = s.W * 256 / D;
    c = (s.tid % L) * (SPLIT ? 4 : 8);
  }
};

// One kernel for each direction, in four forms.  Joint: Q, K and V (parts 0, 1
// and 2, any but one of which may be absent) of a token together, so the angles
// are computed once for both and one barrier serves both sums.  Full: the same
// where all three are there, turned and under a norm over the token, and no
// thread is without channels, which takes every branch out of the row loop
// (when it was added, 480p: 100 instead of 104 us forward, 138 instead of 160 us
// backward).  FullHead: the same under a norm over each head of 128 channels (480p:
// 98 instead of 107 us, 131 instead of 144; heads of 64, which stay with Joint, gain
// nothing from it).
// Single: a part to each blockIdx.y, for parts of different head counts.
enum Form { kSingle, kJoint, kFull, kFullHead };
template <int FORM>
constexpr int turned_parts() {
  return FORM == kSingle ? 1 : 2;
}
template <int FORM>
constexpr int all_parts() {
  return FORM == kSingle ? 1 : 3;
}

// Stages of the ring: with one more the forward of 12 heads takes 109 us instead
// of 96, and that of 40 heads 774 instead of 782.
constexpr int kFwdStages = 2;
// (Two tokens at once, or a joint fp32 row of 640 threads, leave room for two.)
template <typename TX, int THREADS>
constexpr int bwd_stages() {
  return THREADS == 192 || (THREADS == 640 && sizeof(TX) == 4) ? 2 : 3;
}
// Tokens a slot takes at once.
template <int V>
constexpr int fwd_rows() {
  return 2 / V;
}
// CTAs of an SM that the registers are budgeted for.  At 480p two: with three the
// forward takes 111 us instead of 96, with one token at a time and three 98, and
// four 108.  The wide forward too is launched as if two were resident (720p: 782
// us, 830 with a grid for one).
constexpr int kFwdResidents = 2;
// Pieces of one stage, and of a thread's whole ring with the weights behind it.
template <typename TX, int FORM, int V>
constexpr int fwd_pieces() {
  return all_parts<FORM>() * fwd_rows<V>() * V * pieces8<TX>();
}
// (One at a time: 480p 141 instead of 137 us, in fp32 240 instead of 205.  CTAs
// of 640 threads have no registers for two.)
template <int THREADS>
constexpr int bwd_rows() {
  return THREADS == 192 ? 2 : 1;
}
template <typename TX, int FORM, int THREADS>
constexpr int bwd_pieces() {
  return bwd_rows<THREADS>() * bwd_vectors(THREADS) *
         (all_parts<FORM>() + turned_parts<FORM>() * pieces8<TX>());
}
template <typename TX, int FORM, int V>
constexpr int fwd_ring() {
  return kFwdStages * fwd_pieces<TX, FORM, V>() + turned_parts<FORM>() * V * 2;
}
template <typename TX, int FORM, int THREADS>
constexpr int bwd_ring() {
  constexpr int V = bwd_vectors(THREADS);
  return bwd_stages<TX, THREADS>() * bwd_pieces<TX, FORM, THREADS>() + turned_parts<FORM>() * V * 2;
}
constexpr int kAngleBuffers = 2;  // of T tokens (D floats each), for every slot

// A slot's share of the units (at most T tokens of one sample): one of every
// `nslots`, so that the machine is at neighbouring tokens at any time and each
// head's rows are written side by side (480p: 96 and 130 us; with a run of tokens
// to each slot 100 and 137).
struct Share {
  int left, b, n;  // units, and the first one's sample and token
  SPARGE_DEV Share(const HeadsParams& p, int T, int slot, int nslots) {
    const int per_sample = p.span / T;
    const int units = p.M / p.N * per_sample;
    left = slot < units ? (units - slot - 1) / nslots + 1 : 0;
    b = slot / per_sample;
    n = (slot - b * per_sample) * T;
  }
};

template <typename TX, bool INTER, int D, int V, int FORM>
__global__ void __launch_bounds__(row_threads(V), V == 1 ? kFwdResidents : 0) heads_fwd_kernel(
    const __grid_constant__ HeadsParams p) {
  constexpr int T = fwd_rows<V>(), S = kFwdStages, Q8 = pieces8<TX>();
  constexpr int NT = turned_parts<FORM>(), NP = all_parts<FORM>();
  constexpr int STAGE = fwd_pieces<TX, FORM, V>(), RING = fwd_ring<TX, FORM, V>();
  constexpr bool SPLIT = split<TX, INTER>();
  extern __shared__ uint4 smem[];
  __shared__ __align__(16) float red[red_floats(row_threads(V))];
  __shared__ Turns turns;
  constexpr bool FULL = FORM >= kFull;
  const int part0 = FORM == kSingle ? blockIdx.y : 0;
  const HeadsPart& any = p.part[part0];
  const bool plain = FORM == kSingle && any.plain;
  const bool rot = FULL || (p.rotate && !plain);
  const int norm = FORM == kFull       ? SPARGE_HEADS_NORM_TOKEN
                   : FORM == kFullHead ? SPARGE_HEADS_NORM_HEAD
                   : plain             ? 0
                                       : p.norm;
  turns.fill(p);
  Slot s = make_slot(any.W, red, red_half(row_threads(V)));
  __syncthreads();
  const int per_cta = slots_per_cta(any.W);
  if (s.index >= per_cta) return;
  const Place<SPLIT, D, V, FULL> at(s, any.C);
  const int H = any.C / D;
  Share mine(p, T, blockIdx.x * per_cta + s.index, gridDim.x * per_cta);
  if (mine.left == 0) return;

  // Shared memory: the threads' rings, then the slots' angles.
  const Ring ring = {smem + threadIdx.x, static_cast<int>(blockDim.x)};
  const Ring weights = ring + S * STAGE;
  float* ang = reinterpret_cast<float*>(smem + blockDim.x * RING) + s.index * kAngleBuffers * T * D;
  const TX* xp[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const HeadsPart& part = p.part[part0 + i];
    xp[i] = static_cast<const TX*>(part.x) + at.head * part.xs[2] + at.c + mine.b * part.xs[0] +
            mine.n * part.xs[1];
  }
  int ahead_n = mine.n, ahead_left = mine.left;
  const auto issue = [&](Ring stage) {
    if (ahead_left > 0) {
      --ahead_left;
      const bool second = T == 1 || ahead_n + 1 < p.N;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const HeadsPart& part = p.part[part0 + i];
        if (FORM != kJoint || part.x != nullptr) {
#pragma unroll
          for (int t = 0; t < T; ++t) {
#pragma unroll
            for (int v = 0; v < V; ++v)
              if (at.here(v) && (t == 0 || second))
                stage_row<TX, SPLIT, D>(stage + ((i * T + t) * V + v) * Q8,
                                        xp[i] + t * part.xs[1] + v * at.head_step * part.xs[2]);
          }
        }
        xp[i] += part.x_step;
      }
      ahead_n += any.dn;
      if (ahead_n >= p.span) {
        ahead_n -= p.span;
#pragma unroll
        for (int i = 0; i < NP; ++i) xp[i] += p.part[part0 + i].x_wrap;
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < S; ++k) issue(ring + k * STAGE);

#pragma unroll
  for (int i = 0; i < NT; ++i) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int wc = at.c + (norm == 1 ? (at.head + v * at.head_step) * D : 0);
      keep_weight(weights + (i * V + v) * 2,
                  load_weight<INTER, SPLIT, D>(p, norm ? p.part[part0 + i].w : nullptr, at.here(v), wc));
      if (!at.here(v)) {
        // Threads behind the last channel add zeros to the sums.
        for (int k = 0; k < S; ++k) {
          for (int t = 0; t < T; ++t) {
            for (int q = 0; q < Q8; ++q)
              ring[k * STAGE + ((i * T + t) * V + v) * Q8 + q] = make_uint4(0, 0, 0, 0);
          }
        }
      }
    }
  }

  const float inv = 1.f / (norm == 1 ? any.C : D);
  Angles<T, D> angles;
  angles.start(p, any, s, turns, mine.b, mine.n);
  int n = mine.n;
  int64_t out = ((static_cast<int64_t>(mine.b) * H + at.head) * p.N + n) * D + at.c;
  const int64_t far = static_cast<int64_t>(at.head_step) * p.N * D;
  int buf = 0, k = 0;
  for (; mine.left > 0; --mine.left) {
    float* cs = ang + buf * T * D;
    buf ^= 1;
    if (rot) {
      angles.fill(p, s, turns, cs);
      angles.next(p, any, s, turns);
    }
    cp_async_wait<S - 1>();
    const Ring stage = ring + k * STAGE;
    Pairs x[NT * T * V];
    float sums[NT * T * V];
#pragma unroll
    for (int i = 0; i < NT * T * V; ++i) {
      x[i] = unstage_pairs<TX, INTER>(stage + i * Q8);
      sums[i] = dot(x[i], x[i]);
    }
    if (norm == 1) {
      float ts[NT * T];
#pragma unroll
      for (int i = 0; i < NT * T; ++i) {
        ts[i] = sums[i * V];
#pragma unroll
        for (int v = 1; v < V; ++v) ts[i] += sums[i * V + v];
      }
      slot_sum<warp_eights(row_threads(V))>(s, ts);  // its barrier also publishes the angles
#pragma unroll
      for (int i = 0; i < NT * T * V; ++i) sums[i] = ts[i / V];
      if (s.W == 1) slot_sync(s);
    } else {
      if (norm == 2) head_sum<D>(sums);
      if (rot) slot_sync(s);
    }
    const bool second = T == 1 || n + 1 < p.N;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const HeadsPart& part = p.part[part0 + i];
      __nv_bfloat16* y = static_cast<__nv_bfloat16*>(part.y) + out;
#pragma unroll
      for (int t = 0; t < T; ++t) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const bool ok = at.here(v) && (t == 0 || second) && (FORM != kJoint || part.x != nullptr);
          const int q = (i * T + t) * V + v;
          if (i < NT) {
            Pairs u = x[q];
            if (norm) {
              const float r = rsqrtf(sums[q] * inv + p.eps);
              u = mul(mul(u, r), unstage_weight(weights + (i * V + v) * 2));
            }
            if (rot) u = rotate<false, INTER, SPLIT, D>(u, cs + t * D, at.c);
            float f[8];
            from_pairs<INTER>(u, f);
            if (ok) store_row<__nv_bfloat16, SPLIT, D>(y + t * D + v * far, f);
          } else {
            const Raw8<TX> r = unstage8<TX>(stage + q * Q8);
            if (ok) {
              if constexpr (sizeof(TX) == 2) {
                store_row_raw<SPLIT, D>(y + t * D + v * far, r);
              } else {
                float f[8];
                unpack8(r, f);
                store_row<__nv_bfloat16, SPLIT, D>(y + t * D + v * far, f);
              }
            }
          }
        }
      }
    }
    issue(stage);
    k = k + 1 == S ? 0 : k + 1;
    n += any.dn;
    out += any.y_step;
    if (n >= p.span) {
      n -= p.span;
      out += any.y_wrap;
    }
  }
}

template <typename TX, bool INTER, int D, int THREADS, int FORM>
__global__ void __launch_bounds__(THREADS, THREADS == 192 ? 2 : 0) heads_bwd_kernel(
    const __grid_constant__ HeadsParams p) {
  constexpr int V = bwd_vectors(THREADS);
  constexpr int T = bwd_rows<THREADS>(), S = bwd_stages<TX, THREADS>(), Q8 = pieces8<TX>();
  constexpr int NT = turned_parts<FORM>(), NP = all_parts<FORM>();
  constexpr int STAGE = bwd_pieces<TX, FORM, THREADS>(), RING = bwd_ring<TX, FORM, THREADS>();
  constexpr bool SPLIT = split<TX, INTER>();
  constexpr int XAT = NP * T * V;  // the inputs' rows, behind the gradients' rows
  extern __shared__ uint4 smem[];
  constexpr int RED = 2 * NT * T > kSlotRed ? 2 * NT * T : kSlotRed;
  __shared__ __align__(16) float red[red_floats(THREADS, RED)];
  __shared__ Turns turns;
  grid_launch_dependents();
  constexpr bool FULL = FORM >= kFull;
  const int part0 = FORM == kSingle ? blockIdx.y : 0;
  const HeadsPart& any = p.part[part0];
  const bool plain = FORM == kSingle && any.plain;
  const bool rot = FULL || (p.rotate && !plain);
  const int norm = FORM == kFull       ? SPARGE_HEADS_NORM_TOKEN
                   : FORM == kFullHead ? SPARGE_HEADS_NORM_HEAD
                   : plain             ? 0
                                       : p.norm;
  turns.fill(p);
  Slot s = make_slot(any.W, red, red_half(THREADS, RED));
  __syncthreads();
  const int per_cta = slots_per_cta(any.W);
  if (s.index >= per_cta) return;
  const Place<SPLIT, D, V, FULL> at(s, any.C);
  const int H = any.C / D;
  Share mine(p, T, blockIdx.x * per_cta + s.index, gridDim.x * per_cta);

  const Ring ring = {smem + threadIdx.x, static_cast<int>(blockDim.x)};
  const Ring weights = ring + S * STAGE;
  float* ang = reinterpret_cast<float*>(smem + blockDim.x * RING) + s.index * kAngleBuffers * T * D;
  const int64_t far = static_cast<int64_t>(at.head_step) * p.N * D;
  // The places of what is read are computed for each unit: kept like those of the
  // results, their registers spill in the wide kernels (720p, norm per head: 1042
  // us, 1413 with all kept; norm over the token 1078, 1122 with none).
  TX* dx[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const HeadsPart& part = p.part[part0 + i];
    dx[i] = static_cast<TX*>(part.dx) + part_at(part.ds, mine.b, mine.n, at.head, at.c);
  }
  int ahead_b = mine.b, ahead_n = mine.n, ahead_left = mine.left;
  const auto issue = [&](Ring stage) {
    if (ahead_left > 0) {
      --ahead_left;
      const bool second = T == 1 || ahead_n + 1 < p.N;
      const int64_t in = ((static_cast<int64_t>(ahead_b) * H + at.head) * p.N + ahead_n) * D + at.c;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const HeadsPart& part = p.part[part0 + i];
        const TX* x = static_cast<const TX*>(part.x);
        if (i < NT && norm) x += part_at(part.xs, ahead_b, ahead_n, at.head, at.c);
        const bool here = FORM != kJoint || part.y != nullptr;
#pragma unroll
        for (int t = 0; t < T; ++t) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            if (!(here && at.here(v) && (t == 0 || second))) continue;
            const int q = (i * T + t) * V + v;
            stage_row<__nv_bfloat16, SPLIT, D>(
                stage + q, static_cast<const __nv_bfloat16*>(part.y) + in + t * D + v * far);
            if (i < NT && norm)
              stage_row<TX, SPLIT, D>(
                  stage + XAT + q * Q8,
                  x + t * part.xs[1] + v * at.head_step * part.xs[2]);
          }
        }
      }
      any.advance(p.span, ahead_b, ahead_n);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < S; ++k) issue(ring + k * STAGE);

  Pairs dw[NT * V];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int wc = at.c + (norm == 1 ? (at.head + v * at.head_step) * D : 0);
      keep_weight(weights + (i * V + v) * 2,
                  load_weight<INTER, SPLIT, D>(p, norm ? p.part[part0 + i].w : nullptr, at.here(v), wc));
      dw[i * V + v] = {{0, 0}, {0, 0}};
      if (!at.here(v)) {
        for (int k = 0; k < S; ++k) {
          for (int t = 0; t < T; ++t) {
            const int at_row = (i * T + t) * V + v;
            ring[k * STAGE + at_row] = make_uint4(0, 0, 0, 0);
            for (int q = 0; q < Q8; ++q)
              ring[k * STAGE + XAT + at_row * Q8 + q] = make_uint4(0, 0, 0, 0);
          }
        }
      }
    }
  }

  const float inv = 1.f / (norm == 1 ? any.C : D);
  Angles<T, D> angles;
  int n = mine.n, buf = 0;
  if (rot && mine.left > 0) {
    angles.start(p, any, s, turns, mine.b, n);
    angles.fill(p, s, turns, ang);
    angles.next(p, any, s, turns);
    slot_sync(s);
  }
  int k = 0;
  for (; mine.left > 0; --mine.left) {
    cp_async_wait<S - 1>();
    const Ring stage = ring + k * STAGE;
    const float* cs = ang + buf * T * D;
    Pairs g[NT * T * V];
    float sums[2 * NT * T * V];
#pragma unroll
    for (int i = 0; i < NT * T * V; ++i) {
      g[i] = unstage_pairs<__nv_bfloat16, INTER>(stage + i);
      if (rot) g[i] = rotate<true, INTER, SPLIT, D>(g[i], cs + i / V % T * D, at.c);
      if (norm) {
        const Pairs x = unstage_pairs<TX, INTER>(stage + XAT + i * Q8);
        sums[2 * i] = dot(x, x);
        sums[2 * i + 1] = dot(x, mul(g[i], unstage_weight(weights + (i / (T * V) * V + i % V) * 2)));
      }
    }
    // The next token's angles, into the buffer that every warp has read before
    // the barrier of the token before; this token's barrier publishes them.
    buf ^= 1;
    if (rot) {
      angles.fill(p, s, turns, ang + buf * T * D);
      angles.next(p, any, s, turns);
    }
    if (norm == 1) {
      float ts[2 * NT * T];
#pragma unroll
      for (int i = 0; i < 2 * NT * T; ++i) {
        ts[i] = sums[(i / 2) * 2 * V + i % 2];
#pragma unroll
        for (int v = 1; v < V; ++v) ts[i] += sums[((i / 2) * V + v) * 2 + i % 2];
      }
      slot_sum<warp_eights(THREADS)>(s, ts);
#pragma unroll
      for (int i = 0; i < 2 * NT * T * V; ++i) sums[i] = ts[(i / (2 * V)) * 2 + i % 2];
      if (s.W == 1) slot_sync(s);
    } else {
      if (norm == 2) head_sum<D>(sums);
      if (rot) slot_sync(s);
    }
    const bool second = T == 1 || n + 1 < p.N;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const HeadsPart& part = p.part[part0 + i];
#pragma unroll
      for (int t = 0; t < T; ++t) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const bool ok = at.here(v) && (t == 0 || second) && (FORM != kJoint || part.y != nullptr);
          TX* out = dx[i] + t * part.ds[1] + v * at.head_step * part.ds[2];
          const int row = (i * T + t) * V + v;
          if (i < NT) {
            const int q = i < NT ? row : 0;
            Pairs o = g[q];
            if (norm) {
              const float r = rsqrtf(sums[2 * q] * inv + p.eps);
              const Pairs xh = mul(unstage_pairs<TX, INTER>(stage + XAT + q * Q8), r);
              Pairs& to = dw[i < NT ? i * V + v : 0];
              // (A second token behind the sample's end has left-over values.)
              if (t == 0 || second) to = fma(o, xh, to);
              // r (g w - xh mean(g w xh))
              const Pairs w = unstage_weight(weights + (i * V + v) * 2);
              o = mul(fma(xh, -(sums[2 * q + 1] * inv * r), mul(o, w)), r);
            }
            float f[8];
            from_pairs<INTER>(o, f);
            if (ok) store_row<TX, SPLIT, D>(out, f);
          } else {
            const Raw8<__nv_bfloat16> r = unstage8<__nv_bfloat16>(stage + row);
            if (ok) {
              if constexpr (sizeof(TX) == 2) {
                store_row_raw<SPLIT, D>(out, r);
              } else {
                float f[8];
                unpack8(r, f);
                store_row<TX, SPLIT, D>(out, f);
              }
            }
          }
        }
      }
      dx[i] += part.d_step;
    }
    issue(stage);
    k = k + 1 == S ? 0 : k + 1;
    n += any.dn;
    if (n >= p.span) {
      n -= p.span;
#pragma unroll
      for (int i = 0; i < NP; ++i) dx[i] += p.part[part0 + i].d_wrap;
    }
  }
  if (!norm) return;
  // One row of weight sums a CTA: its slots, or with one weight for all heads its
  // warps, add theirs one after the other, in shared memory that the rings no
  // longer need.
  const int warps = per_cta * s.W, warp = s.index * s.W + s.warp;
  const auto cta_sync = [&] { named_barrier_sync(kMaxSlots + 1, warps * 32); };
  float* row = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    float* out = p.part[part0 + i].dw_part;
    if (out == nullptr) continue;
    cta_sync();  // the rings, or the row of the part before, have been read
    if (norm == SPARGE_HEADS_NORM_TOKEN) {
      out += static_cast<int64_t>(blockIdx.x) * any.C;
      for (int turn = 0; turn < per_cta; ++turn) {
        if (turn == s.index) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            if (!at.here(v)) continue;
            float f[8];
            from_pairs<INTER>(dw[i * V + v], f);
            float* to = row + (at.head + v * at.head_step) * D + at.c;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int o = !SPLIT || k < 4 ? k : k - 4 + D / 2;
              if (turn > 0) f[k] += to[o];
              if (turn + 1 < per_cta) to[o] = f[k];
            }
            if (turn + 1 == per_cta) store_row<float, SPLIT, D>(out + (to - row), f);
          }
        }
        if (per_cta > 1) cta_sync();
      }
    } else {
      out += static_cast<int64_t>(blockIdx.x) * D;
      // The heads of the thread, then of the warp.
      float f[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float one[8];
        from_pairs<INTER>(dw[i * V + v], one);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] += at.here(v) ? one[k] : 0.f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
#pragma unroll
        for (int o = D / 8; o < 32; o *= 2) f[k] += __shfl_xor_sync(0xffffffffu, f[k], o);
      }
      for (int turn = 0; turn < warps; ++turn) {
        if (turn == warp && s.lane < D / 8) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int o = at.c + (!SPLIT || k < 4 ? k : k - 4 + D / 2);
            if (turn > 0) f[k] += row[o];
            row[o] = f[k];
          }
          if (turn + 1 == warps) store_row<float, SPLIT, D>(out + at.c, f);
        }
        cta_sync();
      }
    }
  }
}

struct HeadsPlan {
  Form form;
  int built;  // the size of CTA that the kernel is built for
  int V, ctas, threads, slots;  // slots: of a CTA, at most
  int rows;          // tokens that a slot takes at once
  int n;             // parts beside one another in the grid
  int at[3];         // the place of each of the call's parts
  int smem;          // dynamic, of a CTA
  size_t dw_off[3];  // into the workspace
  size_t bytes;
};

template <typename TX, int FORM>
int ring_of_form(const HeadsPlan& pl, bool bwd) {
  if (!bwd) return pl.V == 1 ? fwd_ring<TX, FORM, 1>() : fwd_ring<TX, FORM, 2>();
  return pl.built == 192   ? bwd_ring<TX, FORM, 192>()
         : pl.built == 640 ? bwd_ring<TX, FORM, 640>()
                           : bwd_ring<TX, FORM, 512>();
}
template <typename TX>
int ring_pieces(const HeadsPlan& pl, bool bwd) {
  return pl.form == kSingle ? ring_of_form<TX, kSingle>(pl, bwd) : ring_of_form<TX, kJoint>(pl, bwd);
}
int heads_smem(const HeadsPlan& pl, bool f32, int d, bool bwd) {
  const int pieces = f32 ? ring_pieces<float>(pl, bwd) : ring_pieces<__nv_bfloat16>(pl, bwd);
  return 16 * pieces * pl.threads +
         pl.slots * kAngleBuffers * pl.rows * d * static_cast<int>(sizeof(float));
}

constexpr int kDeclared = 5184;  // shared memory that a kernel declares, at most

HeadsPlan heads_plan(const sparge_heads& a, bool bwd) {
  HeadsPlan pl = {};
  int turned = 0, plain = 0, widest = 0;
  bool same = true;
  for (int i = 0; i < a.n_parts; ++i) {
    const sparge_heads_part& s = a.part[i];
    same = same && s.H == a.part[0].H;
    widest = std::max(widest, s.H * a.d);
    pl.at[i] = s.plain ? 2 : turned;
    (s.plain ? plain : turned)++;
  }
  // Together when the rows are alike: angles and barriers are shared, so 480p
  // takes less time than with a part to each blockIdx.y.
  // Wide rows only where a CTA's ring still fits the shared memory.
  pl.built = bwd ? bwd_threads(widest) : row_threads(row_vectors(widest));
  pl.V = bwd ? bwd_vectors(pl.built) : row_vectors(widest);
  const bool joint = a.n_parts > 1 && same && turned <= 2 && plain <= 1 && turned > 0 &&
                     (pl.V == 1 || (!bwd && a.x_type == SPARGE_BF16));
  const bool full = joint && a.n_parts == 3 && a.rope != nullptr &&
                    (a.norm == SPARGE_HEADS_NORM_TOKEN ||
                     (a.norm == SPARGE_HEADS_NORM_HEAD && a.d == 128)) &&
                    widest % (256 * pl.V) == 0;
  pl.form = !full ? (joint ? kJoint : kSingle)
            : a.norm == SPARGE_HEADS_NORM_TOKEN ? kFull
                                                : kFullHead;
  pl.n = joint ? 1 : a.n_parts;
  int slots_min = kMaxSlots;
  for (int i = 0; i < a.n_parts; ++i) {
    if (!joint) pl.at[i] = i;
    const int W = slot_warps(a.part[i].H * a.d, pl.V);
    pl.threads = std::max(pl.threads, W * slots_per_cta(W) * 32);
    slots_min = std::min(slots_min, slots_per_cta(W));
    pl.slots = std::max(pl.slots, slots_per_cta(W));
  }
  // A grid that is resident as a whole: every CTA stays for its share of the
  // rows.  Shared memory limits it, or registers.
  pl.rows = bwd ? (pl.built == 192 ? 2 : 1) : 2 / pl.V;
  pl.smem = heads_smem(pl, a.x_type == SPARGE_F32, a.d, bwd);
  const int warps = pl.threads / 32;
  const int by_regs = bwd ? resident_warps(bwd_regs(pl.built)) / warps
                          : kFwdResidents * row_threads(pl.V) / pl.threads;
  const int per_sm = std::max(1, std::min(std::min(by_regs, 64 / warps),
                                          kSmemPerSm / (pl.smem + kSmemOfCta + kDeclared)));
  const int64_t units = static_cast<int64_t>(a.B) * ((a.N + pl.rows - 1) / pl.rows);
  const int64_t need = (units + slots_min - 1) / slots_min;
  const int64_t most = (kSMs * per_sm + pl.n - 1) / pl.n;
  pl.ctas = static_cast<int>(std::max<int64_t>(1, std::min(need, most)));
  for (int i = 0; i < a.n_parts; ++i) {
    if (!bwd || a.norm == 0 || a.part[i].plain || a.part[i].dweight == nullptr) continue;
    const int C = a.part[i].H * a.d;
    pl.dw_off[i] = pl.bytes;
    pl.bytes += static_cast<size_t>(pl.ctas) * (a.norm == SPARGE_HEADS_NORM_TOKEN ? C : a.d) *
                sizeof(float);
  }
  return pl;
}

HeadsParams heads_params(const sparge_heads& a, const HeadsPlan& pl) {
  HeadsParams p = {};
  const int per_sample = (a.N + pl.rows - 1) / pl.rows;
  p.span = per_sample * pl.rows;
  const auto shape = [&](HeadsPart& o, int H) {
    o.C = H * a.d;
    o.W = slot_warps(o.C, pl.V);
    const int slots = pl.ctas * slots_per_cta(o.W);
    o.db = slots / per_sample;
    o.dn = slots % per_sample * pl.rows;
    o.y_step = (static_cast<int64_t>(o.db) * H * a.N + o.dn) * a.d;
    o.y_wrap = (static_cast<int64_t>(H) * a.N - p.span) * a.d;
  };
  // An absent part still gives the row its size.
  for (int i = 0; i < 3 && pl.form != kSingle; ++i) shape(p.part[i], a.part[0].H);
  for (int i = 0; i < a.n_parts; ++i) {
    const sparge_heads_part& s = a.part[i];
    HeadsPart& o = p.part[pl.at[i]];
    o.x = s.x;
    o.w = s.weight;
    o.y = s.y;
    o.dx = s.dx;
    for (int k = a.B == 1; k < 3; ++k) o.xs[k] = s.x_stride[k], o.ds[k] = s.dx_stride[k];
    shape(o, s.H);
    o.x_step = o.db * o.xs[0] + o.dn * o.xs[1];
    o.d_step = o.db * o.ds[0] + o.dn * o.ds[1];
    o.x_wrap = o.xs[0] - p.span * o.xs[1];
    o.d_wrap = o.ds[0] - p.span * o.ds[1];
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

// Shared memory of a kernel built for CTAs of THREADS whose slots take T tokens,
// at most: the rings of all its threads and the angles of as many slots as there
// can be.
template <int PIECES, int THREADS, int T, int D>
constexpr int most_smem() {
  constexpr int most = 16 * PIECES * THREADS + kMaxSlots * kAngleBuffers * T * D * 4;
  static_assert(most + kDeclared <= kSmemPerCta, "shared memory of a CTA");
  return most;
}

template <typename TX, bool INTER, int D, int V, int FORM>
cudaError_t launch_fwd_form(const HeadsParams& p, const HeadsPlan& pl, cudaStream_t st) {
  return launch_row_kernel(heads_fwd_kernel<TX, INTER, D, V, FORM>, p, dim3(pl.ctas, pl.n),
                           pl.threads, pl.smem,
                           most_smem<fwd_ring<TX, FORM, V>(), row_threads(V), fwd_rows<V>(), D>(), st);
}

template <typename TX, bool INTER, int D, int V>
cudaError_t launch_fwd(const HeadsParams& p, const HeadsPlan& pl, cudaStream_t st) {
  if constexpr (V == 1 || sizeof(TX) == 2) {
    if (pl.form == kFull) return launch_fwd_form<TX, INTER, D, V, kFull>(p, pl, st);
    if constexpr (D == 128) {
      if (pl.form == kFullHead) return launch_fwd_form<TX, INTER, D, V, kFullHead>(p, pl, st);
    }
    if (pl.form == kJoint) return launch_fwd_form<TX, INTER, D, V, kJoint>(p, pl, st);
  }
  return launch_fwd_form<TX, INTER, D, V, kSingle>(p, pl, st);
}

template <typename TX, bool INTER, int D, int THREADS, int FORM>
cudaError_t launch_bwd_form(const HeadsParams& p, const HeadsPlan& pl, cudaStream_t st) {
  return launch_row_kernel(
      heads_bwd_kernel<TX, INTER, D, THREADS, FORM>, p, dim3(pl.ctas, pl.n), pl.threads, pl.smem,
      most_smem<bwd_ring<TX, FORM, THREADS>(), THREADS, bwd_rows<THREADS>(), D>(), st);
}

template <typename TX, bool INTER, int D, int THREADS>
cudaError_t launch_bwd(const HeadsParams& p, const HeadsPlan& pl, cudaStream_t st) {
  if constexpr (bwd_vectors(THREADS) == 1) {
    if (pl.form == kFull) return launch_bwd_form<TX, INTER, D, THREADS, kFull>(p, pl, st);
    if constexpr (D == 128) {
      if (pl.form == kFullHead) return launch_bwd_form<TX, INTER, D, THREADS, kFullHead>(p, pl, st);
    }
    if (pl.form == kJoint) return launch_bwd_form<TX, INTER, D, THREADS, kJoint>(p, pl, st);
  }
  return launch_bwd_form<TX, INTER, D, THREADS, kSingle>(p, pl, st);
}

template <typename TX, bool INTER, int D>
cudaError_t launch_heads(const HeadsParams& p, const HeadsPlan& pl, bool bwd, cudaStream_t st) {
  if (bwd) {
    if (pl.built == 192) return launch_bwd<TX, INTER, D, 192>(p, pl, st);
    if (pl.built == 640) return launch_bwd<TX, INTER, D, 640>(p, pl, st);
    return launch_bwd<TX, INTER, D, 512>(p, pl, st);
  }
  return pl.V == 1 ? launch_fwd<TX, INTER, D, 1>(p, pl, st) : launch_fwd<TX, INTER, D, 2>(p, pl, st);
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
  if (static_cast<int64_t>(a->B) * a->N > INT32_MAX / 2) return SPARGE_ERR_UNSUPPORTED;
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
      if (normed && s.dweight) HEADS_TRY(check_aligned(s.dweight, 16));
    }
  }
  return SPARGE_OK;
}

Layout layout_of(const void* p, const int64_t (&stride)[3], const sparge_heads& a, int H,
                 int64_t size) {
  return sparge::layout_of(p, {a.B, a.N, H}, stride, a.d * size, size);
}
Layout head_major(const void* p, const sparge_heads& a, int H) {
  const int64_t head = static_cast<int64_t>(a.N) * a.d;
  return layout_of(p, {H * head, a.d, head}, a, H, 2);
}

// Places of a call's tensors: outputs, and what is read beside them.
struct Places {
  int n;
  Layout x[3], y[3], dx[3];
  bool has_x[3];
  Places(const sparge_heads& a, bool bwd) : n(a.n_parts) {
    const int64_t size = a.x_type == SPARGE_F32 ? 4 : 2;
    for (int i = 0; i < n; ++i) {
      const sparge_heads_part& s = a.part[i];
      has_x[i] = !bwd || (a.norm != SPARGE_HEADS_NORM_NONE && !s.plain);
      x[i] = layout_of(s.x, s.x_stride, a, s.H, size);
      y[i] = head_major(s.y, a, s.H);
      dx[i] = layout_of(s.dx, s.dx_stride, a, s.H, size);
    }
  }
  int outputs_apart(bool bwd) const {
    const Layout* out = bwd ? dx : y;
    for (int i = 0; i < n; ++i) {
      if (meets_itself(out[i])) return SPARGE_ERR_INVALID_ARG;
      for (int j = 0; j < i; ++j)
        if (meet(out[i], out[j])) return SPARGE_ERR_INVALID_ARG;
    }
    return SPARGE_OK;
  }
  int inputs_apart(bool bwd) const {
    const Layout* out = bwd ? dx : y;
    for (int i = 0; i < n; ++i) {
      for (int j = 0; j < n; ++j) {
        if (has_x[j] && !(i == j && same_place(out[i], x[j])) && meet(out[i], x[j]))
          return SPARGE_ERR_INVALID_ARG;
        if (bwd && !(i == j && same_place(out[i], y[j])) && meet(out[i], y[j]))
          return SPARGE_ERR_INVALID_ARG;
      }
    }
    return SPARGE_OK;
  }
};

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
  const Places places(*args, false);
  HEADS_TRY(places.outputs_apart(false));
  HEADS_TRY(places.inputs_apart(false));
  const HeadsPlan pl = heads_plan(*args, false);
  return status_of(dispatch_heads(*args, heads_params(*args, pl), pl, false, stream));
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
  const Places places(*args, true);
  HEADS_TRY(places.outputs_apart(true));
  const HeadsPlan pl = heads_plan(*args, true);
  if (pl.bytes > 0) {
    if (workspace == nullptr || ws_bytes < pl.bytes) return SPARGE_ERR_WORKSPACE;
    HEADS_TRY(check_aligned(workspace, 16));
  }
  HEADS_TRY(places.inputs_apart(true));
  HeadsParams p = heads_params(*args, pl);
  ReduceJobs jobs = {};
  for (int i = 0; i < args->n_parts; ++i) {
    const sparge_heads_part& s = args->part[i];
    if (args->norm == SPARGE_HEADS_NORM_NONE || s.plain || s.dweight == nullptr) continue;
    const int C = s.H * args->d;
    float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + pl.dw_off[i]);
    p.part[pl.at[i]].dw_part = part;
    // One row of sums a CTA, of all channels or of those of a head.
    const bool token = args->norm == SPARGE_HEADS_NORM_TOKEN;
    ReduceJob& j = jobs.job[jobs.n++];
    j.src = part;
    j.C = token ? C : args->d;
    j.ld = j.C;
    j.nrow = pl.ctas;
    j.nout = 1;
    j.out = s.dweight;
    j.out_bf16 = args->weight_type == SPARGE_BF16;
  }
  HEADS_TRY(status_of(dispatch_heads(*args, p, pl, true, stream)));
  if (jobs.n > 0) return status_of(launch_reduce_rows(jobs, stream));
  return SPARGE_OK;
}

}  // extern "C"
