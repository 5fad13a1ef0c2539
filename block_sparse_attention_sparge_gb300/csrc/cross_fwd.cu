// Attention over a context on sm_103a: O = softmax(scale Q K^T) V of N query tokens
// over the M tokens of a context, the first kv_len[b] of them valid.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "common.cuh"
#include "cross.cuh"
#include "kernels.h"
#include "rows.cuh"

namespace sparge {

namespace {

constexpr int kBM = kCrossQ;       // queries of a CTA
constexpr int kBN = 64;            // keys of a step
constexpr int kSoftmaxWarps = 4;
constexpr int kProducerWarp = 4;
constexpr int kSWarp = 5;
constexpr int kPVWarp = 6;
constexpr int kFwdThreads = 224;
constexpr int kFwdCtasPerSm = 2;
constexpr float kRescaleLog2 = 8.0f;
constexpr float kLn2 = 0.69314718055994530942f;

template <int D>
struct FwdCfg {
  // K and V stages of 64 keys.  A K stage is held until S of its step, a V
  // stage until PV, so V gets the deeper ring.
  static constexpr int NSK = D == 128 ? 2 : 3;
  static constexpr int NSV = D == 128 ? 3 : 4;
  static constexpr int NP = 2;                        // P phases (the S/P TMEM tiles)
  static constexpr int KCH = D / 64;                  // 128-byte chunks per row
  static constexpr uint32_t kQ = kBM * D * 2;
  static constexpr uint32_t kKV = kBN * D * 2;
  static constexpr uint32_t off_q = 0;
  static constexpr uint32_t off_k = off_q + kQ;
  static constexpr uint32_t off_v = off_k + NSK * kKV;
  static constexpr uint32_t off_bar = off_v + NSV * kKV;
  // barriers
  static constexpr int B_Q = 0;
  static constexpr int B_KF = 1;
  static constexpr int B_VF = B_KF + NSK;
  static constexpr int B_KE = B_VF + NSV;   // K slot free (S of its tile done)
  static constexpr int B_VE = B_KE + NSK;   // V slot free (PV of its tile done)
  static constexpr int B_SF = B_VE + NSV;
  static constexpr int B_PF = B_SF + 2;     // count 128 (all softmax threads)
  static constexpr int B_PV = B_PF + NP;
  static constexpr int B_DRAIN = B_PV + 2;  // count 2 (both issuers)
  static constexpr int NBAR = B_DRAIN + 1;
  static constexpr uint32_t off_tmem_slot = off_bar + NBAR * 8;
  static constexpr uint32_t bytes = off_tmem_slot + 16;
  // The dynamic shared-memory window starts 1024-byte aligned on sm_103a
  // (checked at kernel entry), so no alignment pad is allocated: two CTAs
  // with three V stages then fit one SM.
  static constexpr uint32_t smem_alloc = bytes;
  // S0 [0,64) S1 [64,128) O [128,128+D); P_t (bf16 pairs) over the first 32
  // columns of S_(t & 1).
  static constexpr uint32_t tmem_cols = 256;
  static constexpr uint32_t col_s = 0;
  static constexpr uint32_t col_o = 128;
};


// One launch's tensors beside the tensor maps.
struct CrossFwdParams {
  CrossGeom g;
  HeadsView o;
  float* lse;
  int parts;       // of a query tile's keys
  float* o_part;   // [items, parts, 128, d] where parts > 1
  float* l_part;   // [items, parts, 128]: log2 of the parts' sums
  float scale_log2;
  int32_t* status;
};

template <int D>
__global__ void __launch_bounds__(kFwdThreads, kFwdCtasPerSm)
    cross_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ CrossFwdParams p) {
  using C = FwdCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw;
  const uint32_t s0 = smem_u32(sm);
  if ((s0 & 1023u) != 0u) {  // the swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) report_error(p.status, SPARGE_ERR_CUDA);
    return;
  }
  auto bar = [&](int i) -> uint32_t { return s0 + C::off_bar + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::off_tmem_slot);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int item = blockIdx.x / p.parts, part = blockIdx.x - item * p.parts;
  const int bh = item / p.g.Mq;
  const int qb = item - bh * p.g.Mq;
  const int b = bh / p.g.H, h = bh - b * p.g.H;
  const int hk = h / p.g.group, bk = p.g.Bk > 1 ? b : 0;
  const int len = cross_len(p.g, b);
  // Steps of 64 keys, the part's share of them.
  const int steps = (len + kBN - 1) / kBN;
  const int lo = static_cast<int>(static_cast<int64_t>(steps) * part / p.parts);
  const int n = static_cast<int>(static_cast<int64_t>(steps) * (part + 1) / p.parts) - lo;
  const int N = p.g.N;
  const float scale_log2 = p.scale_log2;
  int32_t* status = p.status;
  auto row_of = [&](int t) -> int { return (lo + t) * kBN; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NBAR; ++i) {
      uint32_t cnt = 1;
      if (i >= C::B_PF && i < C::B_PF + C::NP) cnt = 32 * kSoftmaxWarps;
      if (i == C::B_DRAIN) cnt = 2;
      mbar_init(bar(i), cnt);
    }
    fence_barrier_init();
  }
  if (warp == kSWarp) {
    tmem_alloc(smem_u32(tmem_slot), C::tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    if (lane == 0 && n > 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      mbar_arrive_expect_tx(bar(C::B_Q), C::kQ);
      for (int c = 0; c < C::KCH; ++c)
        tma_load_4d(s0 + C::off_q + c * kBM * 128, &tmQ, bar(C::B_Q), c * 64, qb * kBM, h, b);
      int issued = 0;
      for (int t = 0; t < n; ++t) {
        const int sk = t % C::NSK, sv = t % C::NSV;
        if (t >= C::NSK && !mbar_wait(bar(C::B_KE + sk), ((t / C::NSK) - 1) & 1, kWaitTimeoutNs)) {
          report_error(status, SPARGE_ERR_TIMEOUT);
          break;
        }
        const int rw = row_of(t);
        mbar_arrive_expect_tx(bar(C::B_KF + sk), C::kKV);
        for (int c = 0; c < C::KCH; ++c)
          tma_load_4d(s0 + C::off_k + sk * C::kKV + c * kBN * 128, &tmK, bar(C::B_KF + sk), c * 64,
                      rw, hk, bk);
        if (t >= C::NSV && !mbar_wait(bar(C::B_VE + sv), ((t / C::NSV) - 1) & 1, kWaitTimeoutNs)) {
          report_error(status, SPARGE_ERR_TIMEOUT);
          break;
        }
        mbar_arrive_expect_tx(bar(C::B_VF + sv), C::kKV);
        for (int c = 0; c < C::KCH; ++c)
          tma_load_4d(s0 + C::off_v + sv * C::kKV + c * kBN * 128, &tmV, bar(C::B_VF + sv), c * 64,
                      rw, hk, bk);
        issued = t + 1;
      }
      // Let the last loads land before the CTA can exit (they complete on their own).
      for (int t = max(0, issued - C::NSK); t < issued; ++t)
        mbar_wait(bar(C::B_KF + t % C::NSK), (t / C::NSK) & 1, kWaitTimeoutNs);
      for (int t = max(0, issued - C::NSV); t < issued; ++t)
        mbar_wait(bar(C::B_VF + t % C::NSV), (t / C::NSV) & 1, kWaitTimeoutNs);
    }
  } else if (warp == kSWarp) {
    // ------------------------------------------------------------ S issuer
    // The whole warp runs the loop; one elected lane issues each MMA.
    if (n > 0) {
      constexpr uint32_t idS = idesc_bf16(kBM, kBN, false, false);
      const uint64_t dq0 = sdesc_sw128(s0 + C::off_q, 16, 1024);
      const uint64_t dk0 = sdesc_sw128(s0 + C::off_k, 16, 1024);
      bool ok = warp_wait(bar(C::B_Q), 0);
      for (int t = 0; ok && t < n; ++t) {
        const int s = t % C::NSK;
        // TMEM tile t & 1 holds P(t - 2) until PV(t - 2) has completed.
        if (!warp_wait(bar(C::B_KF + s), (t / C::NSK) & 1) ||
            (t >= 2 && !warp_wait(bar(C::B_PV + (t & 1)), ((t - 2) >> 1) & 1))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t dk = sdesc_add(dk0, s * C::kKV);
        const uint32_t dS = tmem + C::col_s + (t & 1) * kBN;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t koff = (kk & 3) * 32;
          warp_mma_bf16(dS, sdesc_add(dq0, (kk >> 2) * (kBM * 128) + koff),
                        sdesc_add(dk, (kk >> 2) * (kBN * 128) + koff), idS, kk > 0);
        }
        warp_commit(bar(C::B_SF + (t & 1)));
        warp_commit(bar(C::B_KE + s));
      }
      if (!ok && lane == 0) report_error(status, SPARGE_ERR_TIMEOUT);
      // Drain: every MMA this warp issued has completed once this arrives.
      warp_commit(bar(C::B_DRAIN));
      warp_wait(bar(C::B_DRAIN), 0);
    }
  } else if (warp == kPVWarp) {
    // ------------------------------------------------------------ PV issuer
    if (n > 0) {
      constexpr uint32_t idO = idesc_bf16(kBM, D, false, true);
      bool ok = true;
      for (int u = 0; ok && u < n; ++u) {
        const int su = u % C::NSV;
        if (!warp_wait(bar(C::B_VF + su), (u / C::NSV) & 1)) {
          ok = false;
          break;
        }
        // Keys behind the sample's length have P = 0, but their V may hold anything.
        const int valid = len - row_of(u);
        if (valid < kBN)
          zero_tile_rows(sm + C::off_v + su * C::kKV, C::KCH, kBN * 128, valid, kBN, lane);
        if (!warp_wait(bar(C::B_PF + (u % C::NP)), (u / C::NP) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t ap = tmem + C::col_s + (u & 1) * kBN;
        const uint64_t dv = sdesc_sw128(s0 + C::off_v + su * C::kKV, kBN * 128, 1024);
#pragma unroll
        for (int kk = 0; kk < kBN / 16; ++kk)
          warp_mma_bf16_ta(tmem + C::col_o, ap + kk * 8, sdesc_add(dv, kk * 16 * 128), idO,
                           (u > 0 || kk > 0) ? 1u : 0u);
        warp_commit(bar(C::B_VE + su));
        warp_commit(bar(C::B_PV + (u & 1)));
      }
      if (!ok && lane == 0) report_error(status, SPARGE_ERR_TIMEOUT);
      warp_commit(bar(C::B_DRAIN));
      warp_wait(bar(C::B_DRAIN), 0);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int r = threadIdx.x;  // 0..127 == TMEM lane
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const int row = qb * kBM + r;
    float m_used = -INFINITY;
    float l = 0.f;
    bool ok = true;
    // Scores are kept raw; the scale folds into one FFMA before the exp.  The
    // row max is taken on raw scores (the min when the scale is negative).
    const bool pos = scale_log2 > 0.f;
    const float masked = pos ? -INFINITY : INFINITY;
    for (int t = 0; t < n; ++t) {
      if (!warp_wait(bar(C::B_SF + (t & 1)), (t >> 1) & 1)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float x[kBN];
      {
        uint32_t ra[16], rb[16], rc[16], rd[16];
        const uint32_t sa = lane_base + C::col_s + (t & 1) * kBN;
        SPARGE_TMEM_LD_X16(sa + 0, ra);
        SPARGE_TMEM_LD_X16(sa + 16, rb);
        SPARGE_TMEM_LD_X16(sa + 32, rc);
        SPARGE_TMEM_LD_X16(sa + 48, rd);
        SPARGE_TMEM_WAIT_LD16(ra);
        SPARGE_TMEM_WAIT_LD16(rb);
        SPARGE_TMEM_WAIT_LD16(rc);
        SPARGE_TMEM_WAIT_LD16(rd);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          x[c] = __uint_as_float(ra[c]);
          x[16 + c] = __uint_as_float(rb[c]);
          x[32 + c] = __uint_as_float(rc[c]);
          x[48 + c] = __uint_as_float(rd[c]);
        }
      }
      const int valid = len - row_of(t);
      if (valid < kBN) {
#pragma unroll
        for (int c = 0; c < kBN; ++c)
          if (c >= valid) x[c] = masked;
      }
      // Row max as a tree over 8 independent partial maxima, two new
      // columns per three-input max.
      float mp[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) mp[e] = x[e];
      if (pos) {
#pragma unroll
        for (int c = 8; c < 56; c += 16)
#pragma unroll
          for (int e = 0; e < 8; ++e) mp[e] = fmax3(mp[e], x[c + e], x[c + 8 + e]);
#pragma unroll
        for (int e = 0; e < 8; ++e) mp[e] = fmaxf(mp[e], x[56 + e]);
        mp[0] = fmax3(fmax3(mp[0], mp[1], mp[2]), fmax3(mp[3], mp[4], mp[5]), fmaxf(mp[6], mp[7]));
      } else {
#pragma unroll
        for (int c = 8; c < 56; c += 16)
#pragma unroll
          for (int e = 0; e < 8; ++e) mp[e] = fmin3(mp[e], x[c + e], x[c + 8 + e]);
#pragma unroll
        for (int e = 0; e < 8; ++e) mp[e] = fminf(mp[e], x[56 + e]);
        mp[0] = fmin3(fmin3(mp[0], mp[1], mp[2]), fmin3(mp[3], mp[4], mp[5]), fminf(mp[6], mp[7]));
      }
      const float mt = mp[0] * scale_log2;
      const float m_new = fmaxf(m_used, mt);
      // Rescale decision must be warp-uniform (tcgen05.ld/st are warp-wide).
      const bool want = (t > 0) && (m_new - m_used > kRescaleLog2);
      if (t == 0) m_used = m_new;
      if (__any_sync(0xffffffffu, want)) {
        // O holds every PV up to t-1 once that commit has arrived.
        if (!warp_wait(bar(C::B_PV + ((t - 1) & 1)), ((t - 1) >> 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float alpha = want ? exp2f(m_used - m_new) : 1.f;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 16) {
          uint32_t ro[16];
          SPARGE_TMEM_LD_X16(lane_base + C::col_o + c0, ro);
          SPARGE_TMEM_WAIT_LD16(ro);
#pragma unroll
          for (int c = 0; c < 16; ++c) ro[c] = __float_as_uint(__uint_as_float(ro[c]) * alpha);
          SPARGE_TMEM_ST_X16(lane_base + C::col_o + c0, ro);
        }
        tmem_st_wait();
        if (want) {
          l *= alpha;
          m_used = m_new;
        }
      }
      // P_t over the first 32 columns of S_t's tile (this thread's S_t row
      // is already in registers).
      // Eight partial row sums held as four packed pairs; the exponent
      // arguments two columns per packed FMA.
      const uint64_t sl2 = f32x2(scale_log2, scale_log2);
      // (Against a maximum of -inf, scores of -inf would have NaN for 0: any finite
      // reference will do until there is a score.)
      const float ref = m_used == -INFINITY ? 0.f : m_used;
      const uint64_t nm2 = f32x2(-ref, -ref);
      uint64_t rs2[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) rs2[e] = f32x2(0.f, 0.f);
      uint32_t pk[32];
#pragma unroll
      for (int ch = 0; ch < 8; ++ch) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint64_t a = ffma2(f32x2(x[ch * 8 + 2 * e], x[ch * 8 + 2 * e + 1]), sl2, nm2);
          const float p0 = ex2_approx(f32x2_lo(a)), p1 = ex2_approx(f32x2_hi(a));
          rs2[e] = fadd2(rs2[e], f32x2(p0, p1));
          pk[ch * 4 + e] = pack_bf16x2(p0, p1);
        }
      }
      l += ((f32x2_lo(rs2[0]) + f32x2_hi(rs2[0])) + (f32x2_lo(rs2[1]) + f32x2_hi(rs2[1]))) +
           ((f32x2_lo(rs2[2]) + f32x2_hi(rs2[2])) + (f32x2_lo(rs2[3]) + f32x2_hi(rs2[3])));
      {
        const uint32_t pa = lane_base + C::col_s + (t & 1) * kBN;
        SPARGE_TMEM_ST_X16(pa, pk);
        SPARGE_TMEM_ST_X16(pa + 16, (pk + 16));
        tmem_st_wait();
      }
      tc_fence_before();
      mbar_arrive(bar(C::B_PF + (t % C::NP)));
    }
    if (!ok) report_error(status, SPARGE_ERR_TIMEOUT);
    // ---------------------------------------------------------- epilogue
    const bool have = ok && n > 0 && warp_wait(bar(C::B_PV + ((n - 1) & 1)), ((n - 1) >> 1) & 1);
    if (ok && n > 0 && !have) report_error(status, SPARGE_ERR_TIMEOUT);
    tc_fence_after();
    const bool good = have && !(l <= 0.f);  // (a sum that is NaN stays one)
    const float inv_l = good ? 1.f / l : 0.f;
    const bool in_range = row < N;
    const bool split = p.parts > 1;
    __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.o.p) + b * p.o.sb + h * p.o.sh +
                          static_cast<int64_t>(row) * p.o.sn;
    const int64_t prow = (static_cast<int64_t>(item) * p.parts + part) * kBM + r;
    float* opart = p.o_part + prow * D;
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 16) {
      uint32_t ro[16];
      if (have) {
        SPARGE_TMEM_LD_X16(lane_base + C::col_o + c0, ro);
        SPARGE_TMEM_WAIT_LD16(ro);
      } else {
#pragma unroll
        for (int c = 0; c < 16; ++c) ro[c] = 0u;
      }
      float f[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) f[c] = __uint_as_float(ro[c]) * inv_l;
      if (!in_range) continue;
      if (split) {
#pragma unroll
        for (int c = 0; c < 16; c += 4)
          __stcg(reinterpret_cast<float4*>(opart + c0 + c),
                 make_float4(f[c], f[c + 1], f[c + 2], f[c + 3]));
      } else {
        uint32_t w[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) w[c] = pack_bf16x2(f[2 * c], f[2 * c + 1]);
        *reinterpret_cast<uint4*>(orow + c0) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(orow + c0 + 8) = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
    const float l2 = good ? m_used + log2f(l) : -INFINITY;
    if (in_range && split) p.l_part[prow] = l2;
    if (in_range && !split && p.lse != nullptr)
      p.lse[static_cast<int64_t>(bh) * N + row] = l2 * kLn2;
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kSWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::tmem_cols);
  }
}

// Joins the parts of each row: O = sum of 2^(l_p - L) O_p, L = log2 of the sum of
// 2^l_p.  D / 8 threads to a row.
template <int D>
__global__ void __launch_bounds__(256) cross_join_kernel(const __grid_constant__ CrossFwdParams p,
                                                         int64_t rows) {
  constexpr int TPR = D / 8;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * (256 / TPR) + threadIdx.x / TPR;
  const int c = threadIdx.x % TPR * 8;
  if (at >= rows) return;
  const int64_t bh = at / p.g.N;
  const int row = static_cast<int>(at - bh * p.g.N);
  const int64_t item = bh * p.g.Mq + row / kBM;
  const int64_t first = item * p.parts * kBM + row % kBM;
  float top = -INFINITY;
  bool some = false;  // parts with keys; NaN, which the maximum leaves out, is one
  for (int i = 0; i < p.parts; ++i) {
    const float l = __ldg(p.l_part + first + i * kBM);
    top = fmaxf(top, l);
    some |= !(l <= -INFINITY);
  }
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, sum = 0.f;
  if (some) {
    for (int i = 0; i < p.parts; ++i) {
      const float w = exp2f(__ldg(p.l_part + first + i * kBM) - top);
      const float4* src =
          reinterpret_cast<const float4*>(p.o_part + (first + static_cast<int64_t>(i) * kBM) * D + c);
      const float4 a = __ldcg(src), b = __ldcg(src + 1);
      sum += w;
      acc[0] = fmaf(w, a.x, acc[0]), acc[1] = fmaf(w, a.y, acc[1]);
      acc[2] = fmaf(w, a.z, acc[2]), acc[3] = fmaf(w, a.w, acc[3]);
      acc[4] = fmaf(w, b.x, acc[4]), acc[5] = fmaf(w, b.y, acc[5]);
      acc[6] = fmaf(w, b.z, acc[6]), acc[7] = fmaf(w, b.w, acc[7]);
    }
  }
  const float inv = sum <= 0.f ? 0.f : 1.f / sum;
  const int64_t b = bh / p.g.H, h = bh - b * p.g.H;
  __nv_bfloat16* out =
      static_cast<__nv_bfloat16*>(p.o.p) + b * p.o.sb + h * p.o.sh + row * p.o.sn + c;
  *reinterpret_cast<uint4*>(out) =
      make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                 pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
  if (c == 0 && p.lse != nullptr) p.lse[at] = sum <= 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

// Parts of a query tile's keys: one, unless the tiles fill less than half of the
// CTAs that the machine holds; then as many, up to what fills it, as shorten the call,
// where the partial results and their join cost kJoinSteps steps of 64 keys and half of
// one for each part.  (152 tiles, d = 128: 512 keys 12.5 us, in two parts 18.6; 1500
// keys 24.9 and 24.7; at d = 64 10.4 and 12.4, 21.5 and 17.8.)
constexpr int kJoinSteps = 9;
int fwd_parts(const CrossGeom& g) {
  const int64_t items = static_cast<int64_t>(g.B) * g.H * g.Mq, slots = kSMs * kFwdCtasPerSm;
  const int64_t steps = (g.M + kBN - 1) / kBN;
  const int most = static_cast<int>(std::min<int64_t>({slots / items, steps, 64}));
  int best = 1;
  int64_t least = 2 * steps;
  for (int P = 2; P <= most; ++P) {
    const int64_t cost = 2 * ((steps + P - 1) / P) + 2 * kJoinSteps + P;
    if (cost < least) least = cost, best = P;
  }
  return best;
}

template <int D>
cudaError_t launch_fwd_impl(const CrossGeom& g, const sparge_cross& a, void* workspace,
                            cudaStream_t st) {
  using C = FwdCfg<D>;
  CUtensorMap tq, tk, tv;
  if (make_tmap_bf16_4d(&tq, a.q, g.B, g.H, g.N, D, a.q_stride, kBM) != 0 ||
      make_tmap_bf16_4d(&tk, a.k, g.Bk, g.Hk, g.M, D, a.k_stride, kBN) != 0 ||
      make_tmap_bf16_4d(&tv, a.v, g.Bk, g.Hk, g.M, D, a.v_stride, kBN) != 0)
    return cudaErrorInvalidValue;
  const int64_t items = static_cast<int64_t>(g.B) * g.H * g.Mq;
  CrossFwdParams p = {};
  p.g = g;
  p.o = {a.o, a.o_stride[0], a.o_stride[1], a.o_stride[2]};
  p.lse = a.lse;
  p.parts = fwd_parts(g);
  if (p.parts > 1) {
    p.o_part = static_cast<float*>(workspace);
    p.l_part = p.o_part + items * p.parts * kBM * D;
  }
  p.scale_log2 = g.scale * kLog2e;
  p.status = a.status;
  cudaError_t e = cudaFuncSetAttribute(cross_fwd_kernel<D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem_alloc);
  if (e != cudaSuccess) return e;
  cross_fwd_kernel<D><<<static_cast<unsigned>(items * p.parts), kFwdThreads, C::smem_alloc, st>>>(
      tq, tk, tv, p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.parts == 1) return e;
  const int64_t rows = static_cast<int64_t>(g.B) * g.H * g.N, per = 256 / (D / 8);
  cross_join_kernel<D><<<static_cast<unsigned>((rows + per - 1) / per), 256, 0, st>>>(p, rows);
  return cudaGetLastError();
}

// Which form: the persistent one where more query tiles than CTAs fit at once wait
// their turn.  Measured, us, one CTA to a tile / persistent, at 304, 376, 608, 1216 tiles:
//   d = 128, 128 keys   8.1 /  8.9   12.0 / 10.1   14.2 / 11.4   26.6 / 19.8
//            512       13.0 / 14.0   19.6 / 18.9   23.0 / 21.2   43.6 / 36.5
//            1500      25.3 / 26.9   40.1 / 41.8   47.8 / 48.1   92.5 / 88.6
//   d = 64,  128 keys   6.5 /  8.9    9.1 /  9.8   10.8 / 10.8   19.0 / 16.6
//            512       10.7 / 13.6   16.1 / 18.4   18.6 / 20.3   35.2 / 34.2
//            1500      21.5 / 26.3   34.6 / 40.5   40.8 / 45.5   77.9 / 84.4
// At d = 64 a step has half the products for the same softmax, whose chain is what it takes
// (0.78 us a step of two tiles by these times, 0.81 at d = 128), so the persistent form's
// other gains show late and not over long contexts.
bool wide_form(const CrossGeom& g) {
  const int64_t tiles = static_cast<int64_t>(g.B) * g.H * g.Mq;
  return g.d == 128 ? tiles > kFwdCtasPerSm * kSMs : tiles > 4 * kSMs && g.M <= 768;
}

}  // namespace

size_t cross_fwd_workspace_bytes(const CrossGeom& g) {
  const int parts = fwd_parts(g);
  if (parts == 1) return 0;
  return static_cast<size_t>(g.B) * g.H * g.Mq * parts * kBM * (g.d + 1) * sizeof(float);
}

cudaError_t launch_cross_fwd(const CrossGeom& g, const sparge_cross& a, void* workspace,
                             cudaStream_t st) {
  if (wide_form(g)) return launch_cross_fwd_wide(g, a, st);
  return g.d == 128 ? launch_fwd_impl<128>(g, a, workspace, st)
                    : launch_fwd_impl<64>(g, a, workspace, st);
}

}  // namespace sparge
