// Gradients of the attention over a context on sm_103a.
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

constexpr int kBM = kCrossQ;    // queries of a tile
constexpr int kPair = kCrossK;  // keys of a tile

// ---------------------------------------------------------------- D = rowsum(dO * O)
// D / 8 threads to a row, kDeltaRows rows of a head to a thread with all their 16-byte
// loads in flight; one division finds a CTA's head (a row to a thread, found by 64-bit
// divisions: 41 us at 480p, and 34).  The first CTA also starts the item counters of the
// gradient kernels at zero.
constexpr int kDeltaRows = 4;
template <int D>
__global__ void __launch_bounds__(256) cross_delta_kernel(HeadsView o, HeadsView dout, int H, int N,
                                                          int blocks,  // of a head
                                                          float* __restrict__ delta,
                                                          int32_t* __restrict__ work) {
  constexpr int CH = D / 8;      // 16-byte pieces of a row
  constexpr int RPB = 256 / CH;  // rows that a CTA takes at a time
  if (blockIdx.x == 0 && threadIdx.x < 2) work[threadIdx.x] = 0;
  const unsigned bh = blockIdx.x / static_cast<unsigned>(blocks), b = bh / static_cast<unsigned>(H);
  const int64_t h = bh - b * static_cast<unsigned>(H);
  const int first = static_cast<int>(blockIdx.x - bh * blocks) * (RPB * kDeltaRows) + threadIdx.x / CH;
  const int c = threadIdx.x % CH;
  auto at = [&](const HeadsView& v, int n) {
    return reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(v.p) + b * v.sb +
                                          h * v.sh + n * v.sn) + c;
  };
  uint4 x[kDeltaRows], y[kDeltaRows];
#pragma unroll
  for (int i = 0; i < kDeltaRows; ++i) {
    const int n = first + i * RPB;
    x[i] = n < N ? ldg_no_l1(at(o, n)) : make_uint4(0u, 0u, 0u, 0u);
    y[i] = n < N ? ldg_no_l1(at(dout, n)) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < kDeltaRows; ++i) {
    const __nv_bfloat162* hx = reinterpret_cast<const __nv_bfloat162*>(&x[i]);
    const __nv_bfloat162* hy = reinterpret_cast<const __nv_bfloat162*>(&y[i]);
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 fx = __bfloat1622float2(hx[e]), fy = __bfloat1622float2(hy[e]);
      s = fmaf(fx.x, fy.x, s);
      s = fmaf(fx.y, fy.y, s);
    }
#pragma unroll
    for (int off = CH / 2; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    const int n = first + i * RPB;
    if (c == 0 && n < N) delta[static_cast<int64_t>(bh) * N + n] = s;
  }
}

// What is added to a row's scores for its probabilities' exponents: -lse * log2(e); -inf
// for a row without keys (its scores, if any, are all -inf), whose probabilities are 0.
SPARGE_DEV float minus_lse_log2(float lse) { return lse == -INFINITY ? lse : -lse * kLog2e; }

// Loads 32 consecutive fp32 TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32u(uint32_t addr, uint32_t (&a)[16], uint32_t (&b)[16]) {
  SPARGE_TMEM_LD_X16(addr, a);
  SPARGE_TMEM_LD_X16(addr + 16, b);
  SPARGE_TMEM_WAIT_LD16(a);
  SPARGE_TMEM_WAIT_LD16(b);
}

// Warp roles of the gradient kernels: CW compute warps (CW / 4 per TMEM lane
// quarter), then a TMA producer warp, a warp issuing the S and dP MMAs and a
// warp issuing the gradient MMAs.
template <int CW>
struct Roles {
  static constexpr int kCompute = CW;
  static constexpr int kThreads = (CW + 3) * 32;
  static constexpr int kProducer = CW;
  static constexpr int kIssueA = CW + 1;
  static constexpr int kIssueB = CW + 2;
};
constexpr int kDkdvWarps = 8;
constexpr int kDqWarps = 16;

// ---------------------------------------------------------------- dK, dV
template <int D>
struct DkdvCfg {
  // Q and dO arrive per 64-query half of a q-block: a slot holds Q_h and dO_h
  // (64 rows each) and is released once the gradient MMAs of that half are done.
  static constexpr int NSLOT = D == 128 ? 5 : 8;
  static constexpr int NRING = 4;                    // key tiles handed out ahead
  static constexpr uint32_t kKP = kPair * D * 2;     // K (or V) of the 128 keys
  static constexpr uint32_t kQh = 64 * D * 2;        // one Q (or dO) half tile
  static constexpr uint32_t kChunkK = kPair * 128;   // 64-column chunk of the key tile
  static constexpr uint32_t kChunkH = 64 * 128;      // 64-column chunk of a half tile
  static constexpr uint32_t off_k = 0;
  static constexpr uint32_t off_v = off_k + kKP;
  static constexpr uint32_t off_q = off_v + kKP;               // NSLOT Q halves
  static constexpr uint32_t off_do = off_q + NSLOT * kQh;      // NSLOT dO halves
  static constexpr uint32_t off_row = off_do + NSLOT * kQh;    // NSLOT x {-lse*log2e [64], -D [64]}
  static constexpr uint32_t off_info = off_row + NSLOT * 2 * 64 * 4;  // NSLOT x int32
  static constexpr uint32_t off_ring = off_info + 64;          // NRING x {tile, entries}
  static constexpr uint32_t off_bar = off_ring + 64;
  static constexpr int B_KV = 0;              // K/V of a key tile landed
  static constexpr int B_KVE = 1;             // its S^T and dP^T MMAs done: K/V slots free
  static constexpr int B_QF = 2;              // NSLOT, count 32 (producer lanes) + tx
  static constexpr int B_QE = B_QF + NSLOT;   // NSLOT: the half's gradient MMAs done
  // Per query half h, S^T and dP^T are tracked separately, so that P^T and
  // dV of a half proceed while dP^T and dS^T of it are still in flight.
  static constexpr int B_SSF = B_QE + NSLOT;  // 2: S^T_h in TMEM
  static constexpr int B_DPF = B_SSF + 2;     // 2: dP^T_h in TMEM
  static constexpr int B_PPF = B_DPF + 2;     // 2, half h's compute group: P^T_h written
  static constexpr int B_DSF = B_PPF + 2;     // 2, half h's compute group: dS^T_h written
  static constexpr int B_RVF = B_DSF + 2;     // 2: dV MMAs of half h done (S^T_h region free)
  static constexpr int B_RKF = B_RVF + 2;     // 2: dK MMAs of half h done (dP^T_h region free)
  static constexpr int B_DKE = B_RKF + 2;     // all compute threads: dV, dK read out
  static constexpr int B_IF = B_DKE + 1;      // NRING: key tile handed out
  static constexpr int B_IE = B_IF + NRING;   // NRING: read by both issuers and every compute warp
  static constexpr int B_ACC = B_IE + NRING;  // every gradient MMA of a key tile done
  static constexpr int B_DONE = B_ACC + 1;    // count 2
  static constexpr int NBAR = B_DONE + 1;
  static constexpr uint32_t off_slot = off_bar + NBAR * 8;
  static constexpr uint32_t bytes = off_slot + 16;
  // The dynamic shared-memory window starts 1024-byte aligned on sm_103a
  // (checked at kernel entry), so no alignment pad is allocated: five Q/dO
  // slots at d = 128 then fit.
  static constexpr uint32_t smem_alloc = bytes;
  // TMEM: half h of the queries uses columns [128h, 128h + 128): S^T_h at
  // +0 (64 fp32 columns) and dP^T_h at +64.  P^T_h is written over S^T_h as
  // bf16 pairs in chunks of 32 queries: chunk c (queries 32c .. 32c + 31)
  // goes to columns 32c .. 32c + 15, over columns it had read; dS^T_h
  // likewise over dP^T_h.  dV at 256, dK at 256 + 128.
  static constexpr uint32_t tmem_cols = 512;
  static constexpr uint32_t col_dv = 256;
  static constexpr uint32_t col_dk = 384;
};

// One launch's tensors beside the tensor maps.
struct CrossBwdParams {
  CrossGeom g;
  const float* lse;
  float* delta;        // [B, H, N]
  int32_t* work;       // item counters: dQ, dK/dV
  HeadsView dq, dk, dv;
  int q_parts;         // of a query tile's keys
  int k_parts;         // of the query tiles that a key tile sums over
  float* q_part;       // [query tiles, q_parts, 128, d]
  float* k_part;       // [key tiles, k_parts, 128, 2, d]: dV | dK
  float scale, scale_log2;
  int32_t* status;
};

// An item of the dK/dV kernel: a key tile of 128 keys and a share of the query
// tiles that read it (those of the group's heads, and of all samples where they
// share the context).  Key tiles come fastest, so the CTAs that run at the same time
// read the same query tiles, from L2.
struct KeyItem {
  int bk, hk, jt, part;
  int b0;       // first sample
  int lo, hi;   // query tiles, counted through (sample, head of the group, tile)
};
SPARGE_DEV KeyItem key_item(const CrossBwdParams& p, int it) {
  KeyItem x;
  x.jt = it % p.g.Mt;
  it /= p.g.Mt;
  x.part = it % p.k_parts;
  it /= p.k_parts;
  x.hk = it % p.g.Hk;
  x.bk = it / p.g.Hk;
  x.b0 = p.g.Bk > 1 ? x.bk : 0;
  const int64_t all = static_cast<int64_t>(p.g.Bk > 1 ? 1 : p.g.B) * p.g.group * p.g.Mq;
  x.lo = static_cast<int>(all * x.part / p.k_parts);
  x.hi = static_cast<int>(all * (x.part + 1) / p.k_parts);
  return x;
}

// Persistent: one CTA per SM takes items from a counter.  The query tiles of
// successive items share one running count t, which indexes the Q/dO slot ring and
// the barrier phases; the next item's K/V load, S^T and P^T overlap the current
// one's last tiles and epilogue.
template <int D>
__global__ void __launch_bounds__(Roles<kDkdvWarps>::kThreads, 1)
    cross_dkdv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ CUtensorMap tmDO,
                      const __grid_constant__ CrossBwdParams p, int nitems) {
  using C = DkdvCfg<D>;
  using R = Roles<kDkdvWarps>;
  // The dQ kernel (independent of this one) may start on SMs this grid's
  // last CTAs leave idle.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int32_t* status = p.status;
  const int N = p.g.N, M = p.g.M, Mq = p.g.Mq;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw;
  const uint32_t s0 = smem_u32(sm);
  if ((s0 & 1023u) != 0u) {  // the swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) report_error(status, SPARGE_ERR_CUDA);
    return;
  }
  auto bar = [&](int i) -> uint32_t { return s0 + C::off_bar + 8u * i; };
  uint32_t* slot = reinterpret_cast<uint32_t*>(sm + C::off_slot);
  int32_t* info = reinterpret_cast<int32_t*>(sm + C::off_info);
  volatile int32_t* ring = reinterpret_cast<volatile int32_t*>(sm + C::off_ring);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NBAR; ++i) {
      uint32_t cnt = 1;
      if (i >= C::B_QF && i < C::B_QF + C::NSLOT) cnt = 32;
      if (i >= C::B_PPF && i < C::B_PPF + 4) cnt = 32 * R::kCompute / 2;  // PPF, DSF: one half's group
      if (i == C::B_DKE) cnt = 32 * R::kCompute;
      if (i >= C::B_IE && i < C::B_IE + C::NRING) cnt = 2 + R::kCompute;
      if (i == C::B_DONE) cnt = 2;
      mbar_init(bar(i), cnt);
    }
    fence_barrier_init();
  }
  if (warp == R::kIssueA) {
    tmem_alloc(smem_u32(slot), C::tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = slot[0];

  // The seq-th item of this CTA and its number of query tiles, as handed out by
  // the producer through the ring (-1: no more work, -2: the producer gave up).
  auto next_tile = [&](int seq, bool ok, int* n) -> int {
    const int rs = seq % C::NRING;
    if (!ok || !warp_wait(bar(C::B_IF + rs), (seq / C::NRING) & 1)) return -2;
    *n = ring[4 * rs + 1];
    return ring[4 * rs];
  };
  auto release_tile = [&](int seq) { mbar_arrive(bar(C::B_IE + seq % C::NRING)); };
  if (warp == R::kProducer) {
    // ---------------------------------------------------------- producer
    // All 32 lanes: they load the rows' lse and D; lane 0 issues the TMA copies.
    int k = 0, j = 0;  // running counts: halves of query tiles, items with work
    bool ok = true;
    for (int seq = 0;; ++seq) {
      const int rs = seq % C::NRING;
      if (seq >= C::NRING &&
          !mbar_wait(bar(C::B_IE + rs), ((seq / C::NRING) - 1) & 1, kWaitTimeoutNs))
        ok = false;
      ok = __all_sync(0xffffffffu, ok);
      int it = -1;
      if (ok) {
        if (lane == 0) it = atomicAdd(p.work + 1, 1);
        it = __shfl_sync(0xffffffffu, it, 0);
        if (it >= nitems) it = -1;
      }
      KeyItem x{};
      int n = 0;
      const int per = p.g.group * Mq;  // query tiles of a sample
      if (it >= 0) {
        x = key_item(p, it);
        // Samples whose context ends before this tile are left out.
        for (int e = x.lo; e < x.hi;) {
          const int end = min(x.hi, (e / per + 1) * per);
          if (cross_len(p.g, x.b0 + e / per) > x.jt * kPair) n += end - e;
          e = end;
        }
      }
      if (lane == 0) {
        ring[4 * rs] = ok ? it : -2;
        ring[4 * rs + 1] = n;
        mbar_arrive(bar(C::B_IF + rs));
      }
      if (it < 0) break;
      if (n == 0) continue;
      if (j >= 1 && !mbar_wait(bar(C::B_KVE), (j - 1) & 1, kWaitTimeoutNs)) ok = false;
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        continue;  // publishes the failure in the next ring slot, then stops
      }
      const int key0 = x.jt * kPair;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(C::B_KV), 2 * C::kKP);
        for (int c = 0; c < D / 64; ++c) {
          tma_load_4d(s0 + C::off_k + c * C::kChunkK, &tmK, bar(C::B_KV), c * 64, key0, x.hk, x.bk);
          tma_load_4d(s0 + C::off_v + c * C::kChunkK, &tmV, bar(C::B_KV), c * 64, key0, x.hk, x.bk);
        }
      }
      ++j;
      for (int e = x.lo; ok && e < x.hi; ++e) {
        const int b = x.b0 + e / per, h = x.hk * p.g.group + e % per / Mq, i = e % Mq;
        const int valid = min(cross_len(p.g, b) - key0, kPair);  // keys of the tile
        if (valid <= 0) {
          e = (e / per + 1) * per - 1;  // on to the next sample
          continue;
        }
        const float* lse_h = p.lse + (static_cast<int64_t>(b) * p.g.H + h) * N;
        const float* del_h = p.delta + (static_cast<int64_t>(b) * p.g.H + h) * N;
        for (int half = 0; half < 2; ++half, ++k) {
          const int sl = k % C::NSLOT;
          if (k >= C::NSLOT &&
              !mbar_wait(bar(C::B_QE + sl), ((k / C::NSLOT) - 1) & 1, kWaitTimeoutNs))
            ok = false;
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          const int row0 = i * kBM + half * 64;
          if (lane == 0) {
            mbar_expect_tx(bar(C::B_QF + sl), 2 * C::kQh);
            for (int c = 0; c < D / 64; ++c) {
              tma_load_4d(s0 + C::off_q + sl * C::kQh + c * C::kChunkH, &tmQ, bar(C::B_QF + sl),
                          c * 64, row0, h, b);
              tma_load_4d(s0 + C::off_do + sl * C::kQh + c * C::kChunkH, &tmDO,
                          bar(C::B_QF + sl), c * 64, row0, h, b);
            }
            info[sl] = valid;
          }
          // -lse * log2(e) and -D of the half's 64 tokens (queries past N get
          // -inf and 0, so that their P and dS are 0).
          float2 l2, d2;
          const int tok = row0 + lane * 2;
          l2.x = tok < N ? minus_lse_log2(__ldg(lse_h + tok)) : -INFINITY;
          l2.y = tok + 1 < N ? minus_lse_log2(__ldg(lse_h + tok + 1)) : -INFINITY;
          d2.x = tok < N ? -__ldg(del_h + tok) : 0.f;
          d2.y = tok + 1 < N ? -__ldg(del_h + tok + 1) : 0.f;
          float* rowv = reinterpret_cast<float*>(sm + C::off_row + sl * (2 * 64 * 4));
          reinterpret_cast<float2*>(rowv)[lane] = l2;
          reinterpret_cast<float2*>(rowv + 64)[lane] = d2;
          mbar_arrive(bar(C::B_QF + sl));
        }
      }
    }
    if (!ok && lane == 0) report_error(status, SPARGE_ERR_TIMEOUT);
    // Let the last loads land before the CTA can exit.
    if (lane == 0) {
      if (j > 0) mbar_wait(bar(C::B_KV), (j - 1) & 1, kWaitTimeoutNs);
      for (int i = max(0, k - C::NSLOT); i < k; ++i)
        mbar_wait(bar(C::B_QF + i % C::NSLOT), (i / C::NSLOT) & 1, kWaitTimeoutNs);
    }
  } else if (warp == R::kIssueA) {
    // ---------------------------------------------------------- S^T, dP^T
    // S^T_h = K Q_h^T and dP^T_h = V dO_h^T (M = 128 keys, N = 64 queries of
    // half h, K = d).  The whole warp runs the loop; one elected lane issues
    // each MMA.
    constexpr uint32_t idS = idesc_bf16(kPair, 64, false, false);
    const uint64_t dk0 = sdesc_sw128(s0 + C::off_k, 16, 1024);
    const uint64_t dv0 = sdesc_sw128(s0 + C::off_v, 16, 1024);
    bool ok = true;
    int t = 0, j = 0;
    for (int seq = 0;; ++seq) {
      int n = 0;
      const int it = next_tile(seq, ok, &n);
      if (lane == 0) release_tile(seq);
      if (it < 0) {
        if (it == -2) ok = false;
        break;
      }
      if (n == 0) continue;
      if (!warp_wait(bar(C::B_KV), j & 1)) {
        ok = false;
        break;
      }
      ++j;
      for (int e = 0; ok && e < n; ++e, ++t) {
        for (int h = 0; h < 2; ++h) {
          const int k = 2 * t + h, sl = k % C::NSLOT;
          // S^T_h's columns hold P^T_h of entry t - 1 until its dV MMAs are
          // done, dP^T_h's hold dS^T_h until its dK MMAs are.
          if (!warp_wait(bar(C::B_QF + sl), (k / C::NSLOT) & 1) ||
              (t >= 1 && !warp_wait(bar(C::B_RVF + h), (t - 1) & 1))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t dq = sdesc_sw128(s0 + C::off_q + sl * C::kQh, 16, 1024);
          const uint64_t ddo = sdesc_sw128(s0 + C::off_do + sl * C::kQh, 16, 1024);
          const uint32_t dS = tmem + h * 128;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t ka = (kk >> 2) * C::kChunkK + (kk & 3) * 32;
            const uint32_t kb = (kk >> 2) * C::kChunkH + (kk & 3) * 32;
            warp_mma_bf16(dS, sdesc_add(dk0, ka), sdesc_add(dq, kb), idS, kk > 0);
          }
          warp_commit(bar(C::B_SSF + h));
          if (t >= 1 && !warp_wait(bar(C::B_RKF + h), (t - 1) & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t ka = (kk >> 2) * C::kChunkK + (kk & 3) * 32;
            const uint32_t kb = (kk >> 2) * C::kChunkH + (kk & 3) * 32;
            warp_mma_bf16(dS + 64, sdesc_add(dv0, ka), sdesc_add(ddo, kb), idS, kk > 0);
          }
          warp_commit(bar(C::B_DPF + h));
        }
      }
      if (!ok) break;
      warp_commit(bar(C::B_KVE));  // every S^T and dP^T of this tile issued
    }
    if (!ok && lane == 0) report_error(status, SPARGE_ERR_TIMEOUT);
    warp_commit(bar(C::B_DONE));
    warp_wait(bar(C::B_DONE), 0);
  } else if (warp == R::kIssueB) {
    // ---------------------------------------------------------- dV, dK
    // dV += P^T_h dO_h and dK += dS^T_h Q_h (M = 128 keys, N = d, K = the 64
    // queries of half h); A from TMEM, B = dO_h / Q_h read MN-major.  The
    // first MMAs of a tile overwrite the accumulators, after the compute
    // warps have read out the previous tile's.
    constexpr uint32_t idG = idesc_bf16(kPair, D, false, true);
    constexpr int NC = 32;  // queries per P^T / dS^T chunk in TMEM
    bool ok = true;
    int t = 0, j = 0;
    for (int seq = 0;; ++seq) {
      int n = 0;
      const int it = next_tile(seq, ok, &n);
      if (lane == 0) release_tile(seq);
      if (it < 0) {
        if (it == -2) ok = false;
        break;
      }
      if (n == 0) continue;
      for (int e = 0; ok && e < n; ++e, ++t) {
        for (int h = 0; h < 2; ++h) {
          const int sl = (2 * t + h) % C::NSLOT;
          const uint64_t dq = sdesc_sw128(s0 + C::off_q + sl * C::kQh, C::kChunkH, 1024);
          const uint64_t ddo = sdesc_sw128(s0 + C::off_do + sl * C::kQh, C::kChunkH, 1024);
          const uint32_t ap = tmem + h * 128;
          const bool first = e == 0 && h == 0;
          if (!warp_wait(bar(C::B_PPF + h), t & 1) ||
              (first && j >= 1 && !warp_wait(bar(C::B_DKE), (j - 1) & 1))) {
            ok = false;
            break;
          }
          tc_fence_after();
          // Queries 16kk .. 16kk + 15 of the half: the TMEM columns where the
          // compute group wrote their chunk's bf16 pairs.
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            warp_mma_bf16_ta(tmem + C::col_dv, ap + NC * (16 * kk / NC) + (16 * kk % NC) / 2,
                             sdesc_add(ddo, kk * 2048), idG, (!first || kk > 0) ? 1u : 0u);
          warp_commit(bar(C::B_RVF + h));
          if (!warp_wait(bar(C::B_DSF + h), t & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            warp_mma_bf16_ta(tmem + C::col_dk, ap + 64 + NC * (16 * kk / NC) + (16 * kk % NC) / 2,
                             sdesc_add(dq, kk * 2048), idG, (!first || kk > 0) ? 1u : 0u);
          warp_commit(bar(C::B_RKF + h));
          warp_commit(bar(C::B_QE + sl));
        }
      }
      if (!ok) break;
      warp_commit(bar(C::B_ACC));
      ++j;
    }
    if (!ok && lane == 0) report_error(status, SPARGE_ERR_TIMEOUT);
    warp_commit(bar(C::B_DONE));
    warp_wait(bar(C::B_DONE), 0);
  } else if (warp < R::kCompute) {
    // ---------------------------------------------------------- compute
    // Thread = key row r (TMEM lane).  Warp group g = warp / 4 takes query
    // half g of every entry (all 64 queries, in two chunks of 32), so the two
    // warps of an SM sub-partition work on different halves and their
    // latencies overlap (measured at 480p: 1.038 against 1.059 ms per
    // backward with both groups on the same half, 32 queries each).
    constexpr int FPW = D / (R::kCompute / 4);  // features per warp in the epilogue
    const int quarter = warp & 3, cg = warp >> 2;
    const int r = quarter * 32 + lane;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    bool ok = true;
    int t = 0, j = 0;  // entries and tiles with work so far
    for (int seq = 0;; ++seq) {
      int n = 0;
      const int it = next_tile(seq, ok, &n);
      __syncwarp();
      if (lane == 0) release_tile(seq);
      if (it < 0) {
        if (it == -2) ok = false;
        break;
      }
      const KeyItem x = key_item(p, it);
      const int64_t key = static_cast<int64_t>(x.jt) * kPair + r;
      const bool stored = key < M;
      __nv_bfloat16* dk_row = static_cast<__nv_bfloat16*>(p.dk.p) + x.bk * p.dk.sb +
                              x.hk * p.dk.sh + key * p.dk.sn;
      __nv_bfloat16* dv_row = static_cast<__nv_bfloat16*>(p.dv.p) + x.bk * p.dv.sb +
                              x.hk * p.dv.sh + key * p.dv.sn;
      // Partial sums (fp32): dV at [0, d), dK at [d, 2 d) of a row.
      const bool split = p.k_parts > 1;
      const int64_t tile = (static_cast<int64_t>(x.bk) * p.g.Hk + x.hk) * p.g.Mt + x.jt;
      float* part_row = p.k_part + ((tile * p.k_parts + x.part) * kPair + r) * (2 * D);
      if (n == 0) {
        // Keys that no query of this item reads: dK = dV = 0.
        if (stored) {
          const uint4 z = make_uint4(0u, 0u, 0u, 0u);
          for (int cc = cg * FPW; cc < (cg + 1) * FPW; cc += 8) {
            if (split) {
              __stcg(reinterpret_cast<uint4*>(part_row + cc), z);
              __stcg(reinterpret_cast<uint4*>(part_row + cc + 4), z);
              __stcg(reinterpret_cast<uint4*>(part_row + D + cc), z);
              __stcg(reinterpret_cast<uint4*>(part_row + D + cc + 4), z);
            } else {
              *reinterpret_cast<uint4*>(dv_row + cc) = z;
              *reinterpret_cast<uint4*>(dk_row + cc) = z;
            }
          }
        }
        continue;
      }
      for (int e = 0; ok && e < n; ++e, ++t) {
        // This warp group's half of the entry: queries 64h .. 64h + 63 of the
        // q-block, taken in two chunks of 32.
        const int h = cg;
        const int k = 2 * t + h, sl = k % C::NSLOT;
        if (!warp_wait(bar(C::B_QF + sl), (k / C::NSLOT) & 1) ||
            !warp_wait(bar(C::B_SSF + h), t & 1)) {
          ok = false;
          break;
        }
        const int valid = info[sl];
        const bool live = valid > quarter * 32;  // warp-uniform
        const bool key_in = r < valid;
        const float* rowv = reinterpret_cast<const float*>(sm + C::off_row + sl * (2 * 64 * 4));
        tc_fence_after();
        // P^T first (from S^T alone); it is the A operand of dV.  Chunk c's
        // bf16 pairs go over S^T columns 32c .. 32c + 15, which it has read.
        float pr[64];
        const uint64_t sl2 = f32x2(p.scale_log2, p.scale_log2);
#pragma unroll
        for (int c2 = 0; c2 < 2; ++c2) {
          const uint32_t sa = lane_base + h * 128 + 32 * c2;
          uint32_t pk[16];
          if (live) {
            uint32_t sr[2][16];
            SPARGE_TMEM_LD_X16(sa, sr[0]);
            SPARGE_TMEM_LD_X16(sa + 16, sr[1]);
            SPARGE_TMEM_WAIT_LD16(sr[0]);
            SPARGE_TMEM_WAIT_LD16(sr[1]);
            // Two queries per packed instruction: P^T = 2^(S^T * scale*log2e - lse*log2e).
            const ulonglong2* l4 = reinterpret_cast<const ulonglong2*>(rowv + 32 * c2);
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              const ulonglong2 lv = l4[g];  // -lse*log2e of queries 4g .. 4g + 3
#pragma unroll
              for (int q2 = 0; q2 < 2; ++q2) {
                const int col = g * 4 + 2 * q2;
                const uint64_t x = ffma2(f32x2(__uint_as_float(sr[col / 16][col % 16]),
                                               __uint_as_float(sr[col / 16][col % 16 + 1])),
                                         sl2, q2 == 0 ? lv.x : lv.y);
                pr[32 * c2 + col] = key_in ? ex2_approx(f32x2_lo(x)) : 0.f;
                pr[32 * c2 + col + 1] = key_in ? ex2_approx(f32x2_hi(x)) : 0.f;
              }
            }
#pragma unroll
            for (int q4 = 0; q4 < 16; ++q4)
              pk[q4] = pack_bf16x2(pr[32 * c2 + 2 * q4], pr[32 * c2 + 2 * q4 + 1]);
          } else {
#pragma unroll
            for (int q4 = 0; q4 < 32; ++q4) pr[32 * c2 + q4] = 0.f;
#pragma unroll
            for (int q4 = 0; q4 < 16; ++q4) pk[q4] = 0u;
          }
          SPARGE_TMEM_ST_X16(sa, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar(C::B_PPF + h));
        // dS^T = P^T * (dP^T - D).
        if (!warp_wait(bar(C::B_DPF + h), t & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int c2 = 0; c2 < 2; ++c2) {
          const uint32_t sa = lane_base + h * 128 + 32 * c2;
          uint32_t pk[16];
          if (live) {
            uint32_t dr[2][16];
            SPARGE_TMEM_LD_X16(sa + 64, dr[0]);
            SPARGE_TMEM_LD_X16(sa + 64 + 16, dr[1]);
            SPARGE_TMEM_WAIT_LD16(dr[0]);
            SPARGE_TMEM_WAIT_LD16(dr[1]);
            // Two queries per packed instruction.
            const ulonglong2* d4 = reinterpret_cast<const ulonglong2*>(rowv + 64 + 32 * c2);
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              const ulonglong2 dv4 = d4[g];  // -D of queries 4g .. 4g + 3
#pragma unroll
              for (int q2 = 0; q2 < 2; ++q2) {
                const int col = g * 4 + 2 * q2;
                const uint64_t dd = fadd2(f32x2(__uint_as_float(dr[col / 16][col % 16]),
                                                __uint_as_float(dr[col / 16][col % 16 + 1])),
                                          q2 == 0 ? dv4.x : dv4.y);
                const uint64_t z =
                    fmul2(f32x2(pr[32 * c2 + col], pr[32 * c2 + col + 1]), dd);
                // (V behind the sample's length may hold NaN: 0, not 0 * dP.)
                pk[g * 2 + q2] = key_in ? pack_bf16x2(f32x2_lo(z), f32x2_hi(z)) : 0u;
              }
            }
          } else {
#pragma unroll
            for (int q4 = 0; q4 < 16; ++q4) pk[q4] = 0u;
          }
          SPARGE_TMEM_ST_X16(sa + 64, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar(C::B_DSF + h));
      }
      if (!ok) break;
      // Epilogue: lane r holds key r of dV and dK; warp group cg writes its
      // share of the features, then releases the accumulators to the next
      // tile's first MMAs.  A barrier of its own says that the tile's gradient MMAs are
      // done: one phase a tile, each waited for by every warp.  (The halves' barriers
      // would not do: a warp may come here one phase before the last entry's, or when
      // that is over already, and a parity cannot tell these apart.)
      if (!warp_wait(bar(C::B_ACC), j++ & 1)) {
        ok = false;
        break;
      }
      tc_fence_after();
#pragma unroll 1
      for (int cc = cg * FPW; cc < (cg + 1) * FPW; cc += 16) {
        uint32_t rv_[16], rk_[16];
        SPARGE_TMEM_LD_X16(lane_base + C::col_dv + cc, rv_);
        SPARGE_TMEM_LD_X16(lane_base + C::col_dk + cc, rk_);
        SPARGE_TMEM_WAIT_LD16(rv_);
        SPARGE_TMEM_WAIT_LD16(rk_);
        if (cc + 16 >= (cg + 1) * FPW) {
          tc_fence_before();
          mbar_arrive(bar(C::B_DKE));
        }
        if (stored && split) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            __stcg(reinterpret_cast<uint4*>(part_row + cc) + i,
                   make_uint4(rv_[4 * i], rv_[4 * i + 1], rv_[4 * i + 2], rv_[4 * i + 3]));
            __stcg(reinterpret_cast<uint4*>(part_row + D + cc) + i,
                   make_uint4(rk_[4 * i], rk_[4 * i + 1], rk_[4 * i + 2], rk_[4 * i + 3]));
          }
        } else if (stored) {
          uint4 v0, v1, k0, k1;
          v0.x = pack_bf16x2(__uint_as_float(rv_[0]), __uint_as_float(rv_[1]));
          v0.y = pack_bf16x2(__uint_as_float(rv_[2]), __uint_as_float(rv_[3]));
          v0.z = pack_bf16x2(__uint_as_float(rv_[4]), __uint_as_float(rv_[5]));
          v0.w = pack_bf16x2(__uint_as_float(rv_[6]), __uint_as_float(rv_[7]));
          v1.x = pack_bf16x2(__uint_as_float(rv_[8]), __uint_as_float(rv_[9]));
          v1.y = pack_bf16x2(__uint_as_float(rv_[10]), __uint_as_float(rv_[11]));
          v1.z = pack_bf16x2(__uint_as_float(rv_[12]), __uint_as_float(rv_[13]));
          v1.w = pack_bf16x2(__uint_as_float(rv_[14]), __uint_as_float(rv_[15]));
          k0.x = pack_bf16x2(__uint_as_float(rk_[0]) * p.scale, __uint_as_float(rk_[1]) * p.scale);
          k0.y = pack_bf16x2(__uint_as_float(rk_[2]) * p.scale, __uint_as_float(rk_[3]) * p.scale);
          k0.z = pack_bf16x2(__uint_as_float(rk_[4]) * p.scale, __uint_as_float(rk_[5]) * p.scale);
          k0.w = pack_bf16x2(__uint_as_float(rk_[6]) * p.scale, __uint_as_float(rk_[7]) * p.scale);
          k1.x = pack_bf16x2(__uint_as_float(rk_[8]) * p.scale, __uint_as_float(rk_[9]) * p.scale);
          k1.y = pack_bf16x2(__uint_as_float(rk_[10]) * p.scale, __uint_as_float(rk_[11]) * p.scale);
          k1.z = pack_bf16x2(__uint_as_float(rk_[12]) * p.scale, __uint_as_float(rk_[13]) * p.scale);
          k1.w = pack_bf16x2(__uint_as_float(rk_[14]) * p.scale, __uint_as_float(rk_[15]) * p.scale);
          *reinterpret_cast<uint4*>(dv_row + cc) = v0;
          *reinterpret_cast<uint4*>(dv_row + cc + 8) = v1;
          *reinterpret_cast<uint4*>(dk_row + cc) = k0;
          *reinterpret_cast<uint4*>(dk_row + cc + 8) = k1;
        }
      }
    }
    if (!ok) report_error(status, SPARGE_ERR_TIMEOUT);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == R::kIssueA) {
    tc_fence_after();
    tmem_dealloc(tmem, C::tmem_cols);
  }
}

// ---------------------------------------------------------------- dQ
template <int D>
struct DqCfg {
  // K slots outnumber V slots: a K slot is held until dQ of its step, a V
  // slot only until dP.
  static constexpr int NSK = D == 128 ? 3 : 6;
  static constexpr int NSV = D == 128 ? 2 : 4;
  static constexpr int NRING = 4;                   // q-blocks handed out ahead
  static constexpr uint32_t kKP = kPair * D * 2;    // K (or V) of 128 keys
  static constexpr uint32_t kQ = kBM * D * 2;
  static constexpr uint32_t kChunkK = kPair * 128;
  static constexpr uint32_t kChunkQ = kBM * 128;
  static constexpr uint32_t off_q = 0;
  static constexpr uint32_t off_do = off_q + kQ;
  static constexpr uint32_t off_k = off_do + kQ;        // NSK slots of K
  static constexpr uint32_t off_v = off_k + NSK * kKP;  // NSV slots of V
  static constexpr uint32_t off_sum = off_v + NSV * kKP;   // 4 x {sum of P dP [128]}
  static constexpr uint32_t off_ring = off_sum + 4 * kBM * 4;  // NRING q-block ids
  static constexpr uint32_t off_bar = off_ring + 64;
  static constexpr int B_Q = 0;            // Q, dO of a q-block landed
  static constexpr int B_QE = 1;           // its S and dP MMAs done: Q, dO slots free
  static constexpr int B_KF = 2;           // NSK: K landed
  static constexpr int B_VF = B_KF + NSK;  // NSV: V landed
  static constexpr int B_KE = B_VF + NSV;  // NSK: K slot free (dQ of its step done)
  static constexpr int B_VE = B_KE + NSK;  // NSV: V slot free (dP of its step done)
  static constexpr int B_SF = B_VE + NSV;  // 2: S in TMEM buffer b
  static constexpr int B_SE = B_SF + 2;    // 2: dQ read dS of buffer b (buffer free)
  static constexpr int B_DSF = B_SE + 2;   // 8: dS of key chunk c written into buffer b (4b + c)
  static constexpr int B_DPF = B_DSF + 8;  // dP complete
  static constexpr int B_DPE = B_DPF + 1;  // all compute threads: dP read
  static constexpr int B_DQE = B_DPE + 1;  // all compute threads: dQ accumulator read out
  static constexpr int B_IF = B_DQE + 1;   // NRING: q-block id written
  static constexpr int B_IE = B_IF + NRING;  // NRING: id read by both issuers and every compute warp
  static constexpr int B_DS = B_IE + NRING;  // every compute warp: sums of P dP written
  static constexpr int B_DR = B_DS + 1;      // every compute warp: and read
  static constexpr int B_DONE = B_DR + 1;    // count 2
  static constexpr int NBAR = B_DONE + 1;
  static constexpr uint32_t off_slot = off_bar + NBAR * 8;
  static constexpr uint32_t bytes = off_slot + 16;
  // (Starts 1024-byte aligned, see above.)
  static constexpr uint32_t smem_alloc = bytes;
  // TMEM: dQ [0, D), S of step g in buffer g % 2 at 128 + 128 * (g % 2) (128
  // keys; dS of keys 32c .. 32c + 31 written over its columns 32c .. 32c + 15
  // as bf16 pairs), dP at 384.
  static constexpr uint32_t tmem_cols = 512;
  static constexpr uint32_t col_dq = 0;
  static constexpr uint32_t col_s = 128;
  static constexpr uint32_t col_dp = 384;
};

// Persistent: one CTA per SM takes items from a counter: a query tile and a share of
// its sample's key tiles.  Q and dO stay in shared memory as the A operands of S
// and dP; S is double-buffered in TMEM, so S of the next step is computed
// while the compute warps work on this one, and the loads and first MMAs of
// the next item overlap the current one's last steps and epilogue.  The
// steps of successive items share one running step count g, which indexes
// the slot rings and barrier phases.
// OWN: the context is one key tile, so a step has all keys of its rows and D is summed
// here as sum_j P dP, in fp32, and written for the dK/dV kernel, which runs after this
// one; O is not read.  Above kOwnKeys keys D is dO . O of O as the forward rounded it, and a
// row's dS is off by P times what that rounding (and that of P before its product with V)
// makes of D.  With values of mean 0 this shows where few keys are valid: dQ off by 0.0039 in
// the 2-norm with 2 of them, 0.0026 with 10, 0.0024 with 100, which the roundings of dS and of
// the result give alone.  dS depends on the differences of values, but O's rounding on their
// size: where the rows of V share a mean of c times their spread, dQ is off by 0.0037, 0.0088
// and 0.029 for c = 1, 3 and 10 (300 keys, d = 64; 0.0105 and 0.033 for c = 3 and 10 with 2
// valid keys), dK by 0.0029, 0.0057 and 0.019.  Summed here both are off by 0.0024
// throughout.  It costs a longer chain and the overlap of the two kernels (30000 queries
// of 12 heads: 163 -> 185 us at d = 128, 121 -> 145 at d = 64), and with more key tiles a
// pass over S and dP of its own, so up to kOwnKeys keys.
constexpr int kOwnKeys = 64;
template <int D, bool OWN>
__global__ void __launch_bounds__(Roles<kDqWarps>::kThreads, 1)
    cross_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                    const __grid_constant__ CrossBwdParams p, int nitems) {
  using C = DqCfg<D>;
  using R = Roles<kDqWarps>;
  int32_t* status = p.status;
  const int N = p.g.N;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw;
  const uint32_t s0 = smem_u32(sm);
  if ((s0 & 1023u) != 0u) {  // the swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) report_error(status, SPARGE_ERR_CUDA);
    return;
  }
  auto bar = [&](int i) -> uint32_t { return s0 + C::off_bar + 8u * i; };
  uint32_t* slot = reinterpret_cast<uint32_t*>(sm + C::off_slot);
  volatile int32_t* ring = reinterpret_cast<volatile int32_t*>(sm + C::off_ring);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NBAR; ++i) {
      uint32_t cnt = 1;
      if (i == C::B_DPE || i == C::B_DQE) cnt = 32 * R::kCompute;
      if (i >= C::B_DSF && i < C::B_DSF + 8) cnt = 32 * (R::kCompute / 4);
      if (i >= C::B_IE && i < C::B_IE + C::NRING) cnt = 2 + R::kCompute;
      if (i == C::B_DS || i == C::B_DR) cnt = R::kCompute;
      if (i == C::B_DONE) cnt = 2;
      mbar_init(bar(i), cnt);
    }
    fence_barrier_init();
  }
  if (warp == R::kIssueA) {
    tmem_alloc(smem_u32(slot), C::tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;

  // The q-block handed out as the seq-th of this CTA (-1: no more work).  The
  // producer fetches ids from the counter into a ring; the other roles read
  // them from there, in the same order (whole warps: the result is
  // warp-uniform).
  auto next_item = [&](int seq, bool ok) -> int {
    const int rs = seq % C::NRING;
    if (!ok || !warp_wait(bar(C::B_IF + rs), (seq / C::NRING) & 1)) return -2;
    const int it = ring[rs];
    return it;
  };
  auto release_item = [&](int seq) { mbar_arrive(bar(C::B_IE + seq % C::NRING)); };
  struct Item {
    int b, h, qb, part;
    int lo, n;  // first key tile and their number
    int len;    // valid keys of the sample
  };
  auto item_info = [&](int it) -> Item {
    Item x;
    x.part = it % p.q_parts;
    it /= p.q_parts;
    x.qb = it % p.g.Mq;
    it /= p.g.Mq;
    x.h = it % p.g.H;
    x.b = it / p.g.H;
    x.len = cross_len(p.g, x.b);
    const int64_t tiles = (x.len + kPair - 1) / kPair;
    x.lo = static_cast<int>(tiles * x.part / p.q_parts);
    x.n = static_cast<int>(tiles * (x.part + 1) / p.q_parts) - x.lo;
    return x;
  };

  if (warp == R::kProducer) {
    // ---------------------------------------------------------- producer
    if (lane == 0) {
      int g = 0, j = 0;
      bool ok = true;
      for (int seq = 0;; ++seq) {
        const int rs = seq % C::NRING;
        if (seq >= C::NRING &&
            !mbar_wait(bar(C::B_IE + rs), ((seq / C::NRING) - 1) & 1, kWaitTimeoutNs))
          ok = false;
        int it = -1;
        if (ok) {
          const int k = atomicAdd(p.work, 1);
          it = k < nitems ? k : -1;
        }
        ring[rs] = ok ? it : -2;
        mbar_arrive(bar(C::B_IF + rs));
        if (it < 0) break;
        const Item x = item_info(it);
        if (x.n == 0) continue;
        if (j >= 1 && !mbar_wait(bar(C::B_QE), (j - 1) & 1, kWaitTimeoutNs)) {
          ok = false;
          continue;  // publishes the failure in the next ring slot, then stops
        }
        mbar_arrive_expect_tx(bar(C::B_Q), 2 * C::kQ);
        for (int c = 0; c < D / 64; ++c) {
          tma_load_4d(s0 + C::off_q + c * C::kChunkQ, &tmQ, bar(C::B_Q), c * 64, x.qb * kBM, x.h,
                      x.b);
          tma_load_4d(s0 + C::off_do + c * C::kChunkQ, &tmDO, bar(C::B_Q), c * 64, x.qb * kBM,
                      x.h, x.b);
        }
        ++j;
        const int hk = x.h / p.g.group, bk = p.g.Bk > 1 ? x.b : 0;
        for (int u = 0; ok && u < x.n; ++u, ++g) {
          const int sk = g % C::NSK, sv = g % C::NSV, key0 = (x.lo + u) * kPair;
          // K first: S of this step needs it before dP needs V.
          if (g >= C::NSK &&
              !mbar_wait(bar(C::B_KE + sk), ((g / C::NSK) - 1) & 1, kWaitTimeoutNs)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar(C::B_KF + sk), C::kKP);
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(s0 + C::off_k + sk * C::kKP + c * C::kChunkK, &tmK, bar(C::B_KF + sk),
                        c * 64, key0, hk, bk);
          if (g >= C::NSV &&
              !mbar_wait(bar(C::B_VE + sv), ((g / C::NSV) - 1) & 1, kWaitTimeoutNs)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar(C::B_VF + sv), C::kKP);
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(s0 + C::off_v + sv * C::kKP + c * C::kChunkK, &tmV, bar(C::B_VF + sv),
                        c * 64, key0, hk, bk);
        }
      }
      if (!ok) report_error(status, SPARGE_ERR_TIMEOUT);
      // Let the last loads land before the CTA can exit.
      if (j > 0) mbar_wait(bar(C::B_Q), (j - 1) & 1, kWaitTimeoutNs);
      for (int e = max(0, g - C::NSK); e < g; ++e)
        mbar_wait(bar(C::B_KF + e % C::NSK), (e / C::NSK) & 1, kWaitTimeoutNs);
      for (int e = max(0, g - C::NSV); e < g; ++e)
        mbar_wait(bar(C::B_VF + e % C::NSV), (e / C::NSV) & 1, kWaitTimeoutNs);
    }
  } else if (warp == R::kIssueA) {
    // ---------------------------------------------------------- S, dP
    // S_g = Q K_g^T into TMEM buffer g % 2 (free once dQ of step g - 2 has
    // read its dS), then dP_g = dO V_g^T (its region frees once the compute
    // warps have read dP of step g - 1).  M = 128 queries, N = 128 keys.  The
    // whole warp runs the loop; one elected lane issues each MMA.
    constexpr uint32_t idS = idesc_bf16(kBM, kPair, false, false);
    const uint64_t dq0 = sdesc_sw128(s0 + C::off_q, 16, 1024);
    const uint64_t ddo0 = sdesc_sw128(s0 + C::off_do, 16, 1024);
    bool ok = true;
    int g = 0, j = 0;
    for (int seq = 0;; ++seq) {
      const int it = next_item(seq, ok);
      if (lane == 0) release_item(seq);
      if (it < 0) {
        if (it == -2) ok = false;
        break;
      }
      const Item x = item_info(it);
      if (x.n == 0) continue;
      if (!warp_wait(bar(C::B_Q), j & 1)) {
        ok = false;
        break;
      }
      ++j;
      for (int u = 0; ok && u < x.n; ++u, ++g) {
        const int sk = g % C::NSK, sv = g % C::NSV, b = g & 1;
        if (!warp_wait(bar(C::B_KF + sk), (g / C::NSK) & 1) ||
            (g >= 2 && !warp_wait(bar(C::B_SE + b), ((g >> 1) - 1) & 1))) {
          ok = false;
          break;
        }
        // K behind the sample's length may hold anything, and dQ multiplies it by 0.
        const int valid = x.len - (x.lo + u) * kPair;
        if (valid < kPair)
          zero_tile_rows(sm + C::off_k + sk * C::kKP, D / 64, C::kChunkK, valid, kPair, lane);
        tc_fence_after();
        const uint64_t dkd = sdesc_sw128(s0 + C::off_k + sk * C::kKP, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t ka = (kk >> 2) * C::kChunkQ + (kk & 3) * 32;
          const uint32_t kb = (kk >> 2) * C::kChunkK + (kk & 3) * 32;
          warp_mma_bf16(tmem + C::col_s + 128 * b, sdesc_add(dq0, ka), sdesc_add(dkd, kb), idS,
                        kk > 0);
        }
        warp_commit(bar(C::B_SF + b));
        if (!warp_wait(bar(C::B_VF + sv), (g / C::NSV) & 1) ||
            (g >= 1 && !warp_wait(bar(C::B_DPE), (g - 1) & 1))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t dvd = sdesc_sw128(s0 + C::off_v + sv * C::kKP, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t ka = (kk >> 2) * C::kChunkQ + (kk & 3) * 32;
          const uint32_t kb = (kk >> 2) * C::kChunkK + (kk & 3) * 32;
          warp_mma_bf16(tmem + C::col_dp, sdesc_add(ddo0, ka), sdesc_add(dvd, kb), idS, kk > 0);
        }
        warp_commit(bar(C::B_DPF));
        warp_commit(bar(C::B_VE + sv));
      }
      if (!ok) break;
      warp_commit(bar(C::B_QE));  // every S and dP of this q-block issued
    }
    if (!ok && lane == 0) report_error(status, SPARGE_ERR_TIMEOUT);
    warp_commit(bar(C::B_DONE));
    warp_wait(bar(C::B_DONE), 0);
  } else if (warp == R::kIssueB) {
    // ---------------------------------------------------------- dQ
    // dQ += dS_g K_g (A = dS from TMEM buffer g % 2, K = 128 keys; B = the key
    // tile read MN-major, N = d).  dS of keys 16kk .. 16kk + 15 sits in the
    // buffer's columns 32 (kk / 2) + 8 (kk % 2) .. + 7.  The first step of a
    // q-block waits until the previous one's accumulator has been read out.
    constexpr uint32_t idQ = idesc_bf16(kBM, D, false, true);
    bool ok = true;
    int g = 0, j = 0;
    for (int seq = 0;; ++seq) {
      const int it = next_item(seq, ok);
      if (lane == 0) release_item(seq);
      if (it < 0) {
        if (it == -2) ok = false;
        break;
      }
      const Item x = item_info(it);
      if (x.n == 0) continue;
      for (int u = 0; ok && u < x.n; ++u, ++g) {
        const int sk = g % C::NSK, b = g & 1;
        if (u == 0 && j >= 1 && !warp_wait(bar(C::B_DQE), (j - 1) & 1)) {
          ok = false;
          break;
        }
        const uint64_t dkd = sdesc_sw128(s0 + C::off_k + sk * C::kKP, C::kChunkK, 1024);
        const uint32_t ads = tmem + C::col_s + 128 * b;
        // Key chunk c (keys 32c .. 32c + 31) is written by the four warps of
        // group c; its two MMAs start as soon as that chunk is there (measured
        // at 480p: 1.038 against 1.044 ms per backward with one barrier for
        // the whole step).
#pragma unroll
        for (int kk = 0; kk < kPair / 16; ++kk) {
          if ((kk & 1) == 0) {
            if (!warp_wait(bar(C::B_DSF + 4 * b + (kk >> 1)), (g >> 1) & 1)) {
              ok = false;
              break;
            }
            tc_fence_after();
          }
          warp_mma_bf16_ta(tmem + C::col_dq, ads + (kk >> 1) * 32 + (kk & 1) * 8,
                           sdesc_add(dkd, kk * 2048), idQ, (u > 0 || kk > 0) ? 1u : 0u);
        }
        if (!ok) break;
        warp_commit(bar(C::B_SE + b));
        warp_commit(bar(C::B_KE + sk));
      }
      ++j;
    }
    if (!ok && lane == 0) report_error(status, SPARGE_ERR_TIMEOUT);
    warp_commit(bar(C::B_DONE));
    warp_wait(bar(C::B_DONE), 0);
  } else if (warp < R::kCompute) {
    // ---------------------------------------------------------- compute
    // Thread = query row r (TMEM lane); warp group c = warp / 4 takes keys
    // 32c .. 32c + 31 of each step, and features
    // c * D/4 .. (c + 1) * D/4 - 1 of dQ.
    const int quarter = warp & 3, cg = warp >> 2;
    const int r = quarter * 32 + lane;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    bool ok = true;
    int g = 0, seq = 0;
    // The next item, its log-sum-exp and D on their way while this one's epilogue runs
    // (480p 390 -> 373 us for the whole backward).
    int it;
    float lse, delta = 0.f;
    int items = 0;  // that summed D
    float* sums = reinterpret_cast<float*>(sm + C::off_sum);
    auto fetch = [&] {
      it = next_item(seq, ok);
      __syncwarp();
      if (lane == 0) release_item(seq);
      ++seq;
      if (it < 0) return;
      const int rest = it / p.q_parts, n = rest % p.g.Mq * kBM + r;
      const int64_t stat = static_cast<int64_t>(rest / p.g.Mq) * N + n;
      lse = n < N ? __ldg(p.lse + stat) : 0.f;
      if constexpr (!OWN) delta = n < N ? __ldg(p.delta + stat) : 0.f;
    };
    fetch();
    while (true) {
      if (it < 0) {
        if (it == -2) ok = false;
        break;
      }
      const Item x = item_info(it);
      const int row = x.qb * kBM + r;
      const bool rv = row < N;
      __nv_bfloat16* qrow = static_cast<__nv_bfloat16*>(p.dq.p) + x.b * p.dq.sb + x.h * p.dq.sh +
                            static_cast<int64_t>(row) * p.dq.sn;
      const bool split = p.q_parts > 1;
      float* part_row = p.q_part + (static_cast<int64_t>(it) * kBM + r) * D;
      if (x.n == 0) {
        if (rv) {
          const uint4 z = make_uint4(0u, 0u, 0u, 0u);
          for (int cc = cg * (D / 4); cc < (cg + 1) * (D / 4); cc += 8) {
            if (split) {
              __stcg(reinterpret_cast<uint4*>(part_row + cc), z);
              __stcg(reinterpret_cast<uint4*>(part_row + cc + 4), z);
            } else {
              __stcs(reinterpret_cast<uint4*>(qrow + cc), z);
            }
          }
        }
        fetch();
        continue;
      }
      const float nlse2 = minus_lse_log2(lse);
      float drow = delta;
      for (int u = 0; ok && u < x.n; ++u, ++g) {
        const int b = g & 1;
        // Valid keys among this thread's 32 (warp-uniform).
        const int valid = min(32, max(0, x.len - (x.lo + u) * kPair - 32 * cg));
        if (!warp_wait(bar(C::B_SF + b), (g >> 1) & 1) || !warp_wait(bar(C::B_DPF), g & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // dP first, so that its region is released (and dP of the next step
        // computed) while this step's softmax runs.
        uint32_t dr[16], dr2[16], sr[16], sr2[16];
        tmem_ld32u(lane_base + C::col_dp + 32 * cg, dr, dr2);
        tc_fence_before();
        mbar_arrive(bar(C::B_DPE));
        const uint32_t sb = lane_base + C::col_s + 128 * b + 32 * cg;
        tmem_ld32u(sb, sr, sr2);
        uint32_t pk[16];
        if constexpr (OWN) {
          float sum = 0.f;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float pe = ex2_approx(
                fmaf(__uint_as_float(e < 16 ? sr[e] : sr2[e - 16]), p.scale_log2, nlse2));
            sum += e < valid ? pe * __uint_as_float(e < 16 ? dr[e] : dr2[e - 16]) : 0.f;
          }
          // (the last item's sums were read by all)
          if (items > 0 && !warp_wait(bar(C::B_DR), (items - 1) & 1)) {
            ok = false;
            break;
          }
          sums[cg * kBM + r] = sum;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::B_DS));
          if (!warp_wait(bar(C::B_DS), items & 1)) {
            ok = false;
            break;
          }
          drow = (sums[r] + sums[kBM + r]) + (sums[2 * kBM + r] + sums[3 * kBM + r]);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::B_DR));
          ++items;
          if (cg == 0 && rv)
            p.delta[(static_cast<int64_t>(x.b) * p.g.H + x.h) * N + row] = drow;
        }
        if (rv && valid == 32) {
          // Two columns per packed instruction: P = 2^(S * scale*log2e - lse*log2e),
          // dS = P * (dP - D).
          const uint64_t sl2 = f32x2(p.scale_log2, p.scale_log2);
          const uint64_t nl2 = f32x2(nlse2, nlse2);
          const uint64_t nd2 = f32x2(-drow, -drow);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const uint64_t x = ffma2(f32x2(__uint_as_float(e < 16 ? sr[e] : sr2[e - 16]),
                                           __uint_as_float(e < 16 ? sr[e + 1] : sr2[e - 15])),
                                     sl2, nl2);
            const uint64_t pp = f32x2(ex2_approx(f32x2_lo(x)), ex2_approx(f32x2_hi(x)));
            const uint64_t dd = fadd2(f32x2(__uint_as_float(e < 16 ? dr[e] : dr2[e - 16]),
                                            __uint_as_float(e < 16 ? dr[e + 1] : dr2[e - 15])),
                                      nd2);
            const uint64_t z = fmul2(pp, dd);
            pk[e / 2] = pack_bf16x2(f32x2_lo(z), f32x2_hi(z));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float p0 = ex2_approx(
                fmaf(__uint_as_float(e < 16 ? sr[e] : sr2[e - 16]), p.scale_log2, nlse2));
            const float p1 = ex2_approx(
                fmaf(__uint_as_float(e < 16 ? sr[e + 1] : sr2[e - 15]), p.scale_log2, nlse2));
            const float d_a = __uint_as_float(e < 16 ? dr[e] : dr2[e - 16]);
            const float d_b = __uint_as_float(e < 16 ? dr[e + 1] : dr2[e - 15]);
            // (V behind the length may hold NaN: 0, not 0 * dP.)
            pk[e / 2] = pack_bf16x2(rv && e < valid ? p0 * (d_a - drow) : 0.f,
                                    rv && e + 1 < valid ? p1 * (d_b - drow) : 0.f);
          }
        }
        // dS over the first 16 of the 32 S columns this thread read.
        SPARGE_TMEM_ST_X16(sb, pk);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar(C::B_DSF + 4 * b + cg));
      }
      if (!ok) break;
      fetch();
      // Epilogue: read this warp's dQ columns, release the accumulator to the
      // next q-block's dQ MMAs, then scale, convert and store.
      const int gl = g - 1;
      if (!warp_wait(bar(C::B_SE + (gl & 1)), (gl >> 1) & 1)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t ro[D / 4];
#pragma unroll
      for (int c = 0; c < D / 4; c += 16) SPARGE_TMEM_LD_X16(lane_base + C::col_dq + cg * (D / 4) + c, (ro + c));
#pragma unroll
      for (int c = 0; c < D / 4; c += 16) SPARGE_TMEM_WAIT_LD16((ro + c));
      tc_fence_before();
      mbar_arrive(bar(C::B_DQE));
      if (rv && split) {
#pragma unroll
        for (int c = 0; c < D / 4; c += 4)
          __stcg(reinterpret_cast<uint4*>(part_row + cg * (D / 4) + c),
                 make_uint4(ro[c], ro[c + 1], ro[c + 2], ro[c + 3]));
      } else if (rv) {
#pragma unroll
        for (int c = 0; c < D / 4; c += 8) {
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(ro[c + e]) * p.scale;
          __stcs(reinterpret_cast<uint4*>(qrow + cg * (D / 4) + c),
                 make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                            pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])));
        }
      }
    }
    if (!ok) report_error(status, SPARGE_ERR_TIMEOUT);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == R::kIssueA) {
    tc_fence_after();
    tmem_dealloc(tmem, C::tmem_cols);
    // Started early beside the dK/dV grid: the grid completes only after that
    // one has, so work after this call sees dK and dV written.
    if (blockIdx.x == 0 && threadIdx.x == R::kIssueA * 32)
      asm volatile("griddepcontrol.wait;" ::: "memory");
  }
}

// Sums of the parts, in their order: dV | dK of the key tiles, dQ of the query
// tiles.  A thread takes eight values of a row; there are parts only where tiles are few
// for the machine, so 32 bits count the threads.
template <int D>
__global__ void __launch_bounds__(256) cross_sum_kernel(const __grid_constant__ CrossBwdParams p,
                                                        uint32_t key_work, uint32_t query_work) {
  constexpr uint32_t TPR = D / 8;
  uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= key_work + query_work) return;
  const bool keys = i < key_work;
  if (!keys) i -= key_work;
  const int c = static_cast<int>(i % TPR) * 8;
  i /= TPR;
  const int which = keys ? static_cast<int>(i & 1) : 0;  // dV, dK
  if (keys) i >>= 1;
  const uint32_t len = keys ? p.g.M : p.g.N, heads = keys ? p.g.Hk : p.g.H;
  const int tiles = keys ? p.g.Mt : p.g.Mq, parts = keys ? p.k_parts : p.q_parts;
  const uint32_t bh = i / len;
  const int64_t n = i - bh * len, b = bh / heads, h = bh % heads;
  const int64_t tile = static_cast<int64_t>(bh) * tiles + n / kPair;
  const int width = keys ? 2 * D : D;
  const float* src = (keys ? p.k_part : p.q_part) + (tile * parts * kPair + n % kPair) * width +
                     which * D + c;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int q = 0; q < parts; ++q) {
    const float4* s = reinterpret_cast<const float4*>(src + static_cast<int64_t>(q) * kPair * width);
    const float4 x = __ldcg(s), y = __ldcg(s + 1);
    acc[0] += x.x, acc[1] += x.y, acc[2] += x.z, acc[3] += x.w;
    acc[4] += y.x, acc[5] += y.y, acc[6] += y.z, acc[7] += y.w;
  }
  const HeadsView& v = keys ? (which ? p.dk : p.dv) : p.dq;
  const float f = keys && !which ? 1.f : p.scale;
  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(v.p) + b * v.sb + h * v.sh + n * v.sn + c) =
      make_uint4(pack_bf16x2(acc[0] * f, acc[1] * f), pack_bf16x2(acc[2] * f, acc[3] * f),
                 pack_bf16x2(acc[4] * f, acc[5] * f), pack_bf16x2(acc[6] * f, acc[7] * f));
}

// Parts of the query tiles that a key tile sums over: as many as make the grid's
// waves short, where a part costs kPartCost query tiles' time beside its own (the
// K and V load, the partial sums and their join).
constexpr int kPartCost = 3, kMaxParts = 64;
int key_parts(const CrossGeom& g) {
  const int64_t tiles = static_cast<int64_t>(g.Bk) * g.Hk * g.Mt;
  const int64_t all = static_cast<int64_t>(g.Bk > 1 ? 1 : g.B) * g.group * g.Mq;
  int best = 1;
  int64_t least = INT64_MAX;
  for (int P = 1; P <= kMaxParts && P <= all && (P == 1 || tiles * P <= 16 * kSMs); ++P) {
    const int64_t waves = (tiles * P + kSMs - 1) / kSMs;
    const int64_t cost = waves * ((all + P - 1) / P + (P > 1 ? kPartCost : 1));
    if (cost < least) least = cost, best = P;
  }
  return best;
}
// Parts of a query tile's key tiles: one, unless the query tiles fill less than
// half of the machine; then as many as fill it, of two tiles at least.
int query_parts(const CrossGeom& g) {
  const int64_t tiles = static_cast<int64_t>(g.B) * g.H * g.Mq;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({kSMs / tiles, g.Mt / 2, kMaxParts})));
}

// Workspace: D, the counters, partial dV | dK and dQ.
struct Workspace {
  size_t delta, work, k_part, q_part, bytes;
};
Workspace workspace_of(const CrossGeom& g) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const int kp = key_parts(g), qp = query_parts(g);
  Workspace w = {};
  w.work = up(static_cast<size_t>(g.B) * g.H * g.N * sizeof(float));
  w.k_part = w.work + up(2 * sizeof(int32_t));
  w.q_part = w.k_part +
             (kp > 1 ? static_cast<size_t>(g.Bk) * g.Hk * g.Mt * kp * kPair * 2 * g.d * sizeof(float) : 0);
  w.bytes = w.q_part +
            (qp > 1 ? static_cast<size_t>(g.B) * g.H * g.Mq * qp * kBM * g.d * sizeof(float) : 0);
  return w;
}

template <int D>
cudaError_t launch_bwd_impl(const CrossGeom& g, const sparge_cross& a, void* workspace,
                            cudaStream_t st) {
  const Workspace w = workspace_of(g);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  auto view = [](const void* p, const int64_t (&s)[3]) {
    return HeadsView{const_cast<void*>(p), s[0], s[1], s[2]};
  };
  float* delta = reinterpret_cast<float*>(ws + w.delta);
  CrossBwdParams p = {};
  p.g = g;
  p.lse = a.lse;
  p.delta = delta;
  p.work = reinterpret_cast<int32_t*>(ws + w.work);
  p.dq = view(a.dq, a.dq_stride);
  p.dk = view(a.dk, a.dk_stride);
  p.dv = view(a.dv, a.dv_stride);
  p.q_parts = query_parts(g);
  p.k_parts = key_parts(g);
  p.k_part = reinterpret_cast<float*>(ws + w.k_part);
  p.q_part = reinterpret_cast<float*>(ws + w.q_part);
  p.scale = g.scale;
  p.scale_log2 = g.scale * kLog2e;
  p.status = a.status;
  // Q and dO in 128-row boxes for the dQ kernel, in 64-row boxes (query halves) for
  // the dK/dV kernel.
  CUtensorMap tq, tk, tv, tdo, tq64, tdo64;
  if (make_tmap_bf16_4d(&tq, a.q, g.B, g.H, g.N, D, a.q_stride, kBM) != 0 ||
      make_tmap_bf16_4d(&tdo, a.dout, g.B, g.H, g.N, D, a.dout_stride, kBM) != 0 ||
      make_tmap_bf16_4d(&tq64, a.q, g.B, g.H, g.N, D, a.q_stride, 64) != 0 ||
      make_tmap_bf16_4d(&tdo64, a.dout, g.B, g.H, g.N, D, a.dout_stride, 64) != 0 ||
      make_tmap_bf16_4d(&tk, a.k, g.Bk, g.Hk, g.M, D, a.k_stride, kPair) != 0 ||
      make_tmap_bf16_4d(&tv, a.v, g.Bk, g.Hk, g.M, D, a.v_stride, kPair) != 0)
    return cudaErrorInvalidValue;

  // Few keys: D is the dQ kernel's, which runs first.
  const bool own = g.M <= kOwnKeys;
  cudaError_t e;
  if (own) {
    e = cudaMemsetAsync(p.work, 0, 2 * sizeof(int32_t), st);
  } else {
    const int per = 256 / (D / 8) * kDeltaRows, blocks = (g.N + per - 1) / per;
    cross_delta_kernel<D><<<static_cast<unsigned>(g.B) * g.H * blocks, 256, 0, st>>>(
        view(a.o, a.o_stride), view(a.dout, a.dout_stride), g.H, g.N, blocks, delta, p.work);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;

  // Both gradient kernels are persistent: one CTA per SM (or per item when there
  // are fewer), taking items from their counters.
  auto run_dkdv = [&]() -> cudaError_t {
    const int k_items = g.Bk * g.Hk * g.Mt * p.k_parts;
    const cudaError_t r = cudaFuncSetAttribute(
        cross_dkdv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, DkdvCfg<D>::smem_alloc);
    if (r != cudaSuccess) return r;
    cross_dkdv_kernel<D><<<std::min(k_items, kSMs), Roles<kDkdvWarps>::kThreads,
                           DkdvCfg<D>::smem_alloc, st>>>(tq64, tk, tv, tdo64, p, k_items);
    return cudaGetLastError();
  };
  auto run_dq = [&](auto* kernel) -> cudaError_t {
    const int q_items = g.B * g.H * g.Mq * p.q_parts;
    const cudaError_t r = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, DqCfg<D>::smem_alloc);
    if (r != cudaSuccess) return r;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(std::min(q_items, kSMs));
    cfg.blockDim = dim3(Roles<kDqWarps>::kThreads);
    cfg.dynamicSmemBytes = DqCfg<D>::smem_alloc;
    cfg.stream = st;
    // Programmatic dependent launch: the dQ CTAs may start while the last dK/dV
    // CTAs run (D and the counters were complete before dK/dV started).
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = own ? 0 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, tq, tk, tv, tdo, p, q_items);
  };
  e = own ? run_dq(cross_dq_kernel<D, true>) : run_dkdv();
  if (e != cudaSuccess) return e;
  e = own ? run_dkdv() : run_dq(cross_dq_kernel<D, false>);
  if (e != cudaSuccess) return e;

  const int64_t key_work = p.k_parts > 1 ? static_cast<int64_t>(g.Bk) * g.Hk * g.M * 2 * (D / 8) : 0;
  const int64_t query_work =
      p.q_parts > 1 ? static_cast<int64_t>(g.B) * g.H * g.N * (D / 8) : 0;
  if (key_work + query_work == 0) return cudaSuccess;
  cross_sum_kernel<D><<<static_cast<unsigned>((key_work + query_work + 255) / 256), 256, 0, st>>>(
      p, static_cast<uint32_t>(key_work), static_cast<uint32_t>(query_work));
  return cudaGetLastError();
}

}  // namespace

size_t cross_bwd_workspace_bytes(const CrossGeom& g) { return workspace_of(g).bytes; }

cudaError_t launch_cross_bwd(const CrossGeom& g, const sparge_cross& a, void* workspace,
                             cudaStream_t st) {
  return g.d == 128 ? launch_bwd_impl<128>(g, a, workspace, st)
                    : launch_bwd_impl<64>(g, a, workspace, st);
}

}  // namespace sparge
