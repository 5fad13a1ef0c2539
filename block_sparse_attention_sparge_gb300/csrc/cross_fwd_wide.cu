// Attention over a context on sm_103a where the query tiles fill the machine: O =
// softmax(scale Q K^T) V, the first kv_len[b] of M keys valid.
//
// Persistent, one CTA an SM.  A CTA works on two tiles of 128 queries that read the
// same keys (of one head, or of two heads of a group) in steps of 64 keys, with two S
// tiles to each (4 x 64 columns of tensor memory, and 2 x d for the outputs: all 512 at
// d = 128).  A warp to a tile issues its products, S two steps ahead of PV, where the
// step after an item's last is the next item's first: the pipe does not drain between
// items, whose queries come into a second buffer meanwhile.  A thread's products run in
// their order and a commit stands for all of them so far, so S(t + 2) takes the place of
// P(t), and its being there means that PV(t) is.  (One warp for both tiles spent 4600
// cycles a step of 128 keys on issuing 2080 cycles of products.)
//
// Softmax (a thread to a row): the exponents are taken against the maximum that the row
// had before the step, in one pass over the step's scores, which also finds whether one
// of them passes it by more than 2^8.  Only then (and in the first step) the maximum
// moves, sum and output are rescaled and the pass is repeated; the results are exact
// either way, because sum and output share the reference.  A maximum of -inf (all scores
// so far) stands for no reference: the pass takes 0, and moves to the first score that is
// there, however small.
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

constexpr int kBM = kCrossQ;  // queries of a tile
constexpr int kBN = 64;       // keys of a step
// Warps: softmax (four to a tile), output (four), producer, issuers (one to a tile).
constexpr int kOutput = 8, kProducer = 12, kIssuer = 13;
constexpr int kThreads = 15 * 32;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kSlack = 8.f;  // log2 of what a score may pass the reference by

template <int D>
struct WideCfg {
  static constexpr int KCH = D / 64;             // 128-byte chunks of a row
  static constexpr int NS = D == 128 ? 6 : 12;   // slots of a step's keys or values
  static constexpr uint32_t kQ = kBM * D * 2;    // of one tile
  static constexpr uint32_t kKV = kBN * D * 2;
  static constexpr uint32_t off_q = 0;           // two buffers of two tiles
  static constexpr uint32_t off_kv = off_q + 4 * kQ;
  static constexpr uint32_t off_bar = off_kv + NS * kKV;
  static constexpr int B_QF = 0;            // 2: an item's queries landed
  static constexpr int B_QE = 2;            // 2: its S products done, its output (put in
                                            // the queries' place) stored by four warps
  static constexpr int B_F = 4;             // NS: keys or values landed
  static constexpr int B_E = B_F + NS;      // NS: their products done
  static constexpr int B_S = B_E + NS;      // 2 tiles x 2 steps: S there (and every
                                            // product before)
  static constexpr int B_P = B_S + 4;       // the same, 128 threads: P written
  static constexpr int B_PV = B_P + 4;      // 2: a step's PV done
  static constexpr int B_O = B_PV + 2;      // 2: an item's O complete
  static constexpr int B_L = B_O + 2;       // 2, 128 threads: its rows' sums written
  static constexpr int B_OE = B_L + 2;      // 2, 128 threads: O and the sums read
  static constexpr int B_Z = B_OE + 2;      // NS: V behind a sample's length zeroed
  static constexpr int B_DONE = B_Z + NS;
  static constexpr int NBAR = B_DONE + 1;
  static constexpr uint32_t off_slot = off_bar + NBAR * 8;
  static constexpr uint32_t off_word = off_slot + 16;  // a word of each slot
  static constexpr uint32_t off_row = off_word + NS * 4;  // reference and sum of each row
  static constexpr uint32_t bytes = off_row + 2 * kBM * 8;
  static constexpr uint32_t col_o = 256;
};

struct WideParams {
  CrossGeom g;
  HeadsView o;
  float* lse;
  float scale_log2;
  int even;       // query tiles of a key head, rounded up to pairs
  int tiles;      // of all key heads and samples
  int spread;     // pairs dealt out one by one (contexts of different lengths)
  int32_t* status;
};

// The items of a CTA: pairs of query tiles, a share of neighbouring ones, or every
// n-th where the contexts' lengths differ.
struct Item {
  int b, hk, v, n;  // sample, key head, first tile of the head's, tiles (1 or 2)
  int len, steps;
};
struct Walk {
  int at, end, step;
  SPARGE_DEV explicit Walk(const WideParams& p) {
    if (p.spread) {
      at = 2 * blockIdx.x;
      end = p.tiles;
      step = 2 * gridDim.x;
    } else {
      at = static_cast<int>(static_cast<int64_t>(p.tiles) * blockIdx.x / gridDim.x);
      end = static_cast<int>(static_cast<int64_t>(p.tiles) * (blockIdx.x + 1) / gridDim.x);
      step = 0;
    }
  }
  // The next item; false behind the last.
  SPARGE_DEV bool next(const WideParams& p, Item& x) {
    const int own = p.g.group * p.g.Mq;  // tiles of a key head that are there
    while (at < end) {
      const int bh = static_cast<unsigned>(at) / static_cast<unsigned>(p.even);
      x.v = at - bh * p.even;
      x.n = min(min(2, own - x.v), end - at);
      at = step > 0 ? (at > end - step ? end : at + step) : at + min(2, min(p.even - x.v, end - at));
      if (x.n <= 0) continue;  // the pair's empty half
      x.b = static_cast<unsigned>(bh) / static_cast<unsigned>(p.g.Hk);
      x.hk = bh - x.b * p.g.Hk;
      x.len = cross_len(p.g, x.b);
      x.steps = (x.len + kBN - 1) / kBN;
      return true;
    }
    return false;
  }
  // The head and first query of an item's i-th tile.
  SPARGE_DEV void tile(const WideParams& p, const Item& x, int i, int& h, int& row) const {
    const int g = static_cast<unsigned>(x.v + i) / static_cast<unsigned>(p.g.Mq);
    h = x.hk * p.g.group + g;
    row = (x.v + i - g * p.g.Mq) * kBM;
  }
};

// What the issuers are told of a step, with its keys: its tiles, whether it is an item's
// first or last, the item's query buffer, and its valid keys where V has to be zeroed
// behind them (else all).  0: no more steps.
SPARGE_DEV int step_word(const Item& x, int t, int items, int M) {
  const int valid = x.len - t * kBN;
  return x.n | (t == 0 ? 4 : 0) | (t == x.steps - 1 ? 8 : 0) | (items & 1) << 4 |
         (valid < kBN && x.len < M ? valid : kBN) << 8;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    cross_fwd_wide_kernel(const __grid_constant__ CUtensorMap tmQ,
                          const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ CUtensorMap tmO,
                          const __grid_constant__ WideParams p) {
  using C = WideCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw;
  const uint32_t s0 = smem_u32(sm);
  if ((s0 & 1023u) != 0u) {  // the swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) report_error(p.status, SPARGE_ERR_CUDA);
    return;
  }
  auto bar = [&](int i) -> uint32_t { return s0 + C::off_bar + 8u * i; };
  uint32_t* slot = reinterpret_cast<uint32_t*>(sm + C::off_slot);
  volatile int32_t* words = reinterpret_cast<volatile int32_t*>(sm + C::off_word);
  // (The shuffles tell the compiler that these are the same in all lanes, so what the
  // issuers compute from them stays in uniform registers: 60 instead of 30 cycles for
  // each MMA otherwise.)
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NBAR; ++i) {
      uint32_t count = 1;
      if ((i >= C::B_P && i < C::B_P + 4) || (i >= C::B_L && i < C::B_OE + 2)) count = 128;
      if (i == C::B_QE || i == C::B_QE + 1) count = 2 + 4;
      if ((i >= C::B_E && i < C::B_E + C::NS) || i == C::B_DONE) count = 2;
      mbar_init(bar(i), count);
    }
    fence_barrier_init();
  }
  if (warp == kIssuer) {
    tmem_alloc(smem_u32(slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *slot, 0);

  if (warp == kProducer) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      bool ok = true;
      int g = 0, items = 0;  // tiles of keys and values; items
      auto slot_of = [&]() -> int {
        const int sl = g % C::NS;
        if (ok && g >= C::NS && !mbar_wait(bar(C::B_E + sl), ((g / C::NS) - 1) & 1, kWaitTimeoutNs))
          ok = false;
        return sl;
      };
      auto load = [&](const CUtensorMap* map, const Item& x, int t, int word) {
        const int sl = slot_of();
        if (!ok) return;
        words[sl] = word;
        mbar_arrive_expect_tx(bar(C::B_F + sl), C::kKV);
        for (int c = 0; c < C::KCH; ++c)
          tma_load_4d(s0 + C::off_kv + sl * C::kKV + c * kBN * 128, map, bar(C::B_F + sl), c * 64,
                      t * kBN, x.hk, p.g.Bk > 1 ? x.b : 0);
        ++g;
      };
      Walk walk(p);
      for (Item x; ok && walk.next(p, x);) {
        if (x.steps == 0) continue;
        const int qb = items & 1;
        if (items >= 2 && !mbar_wait(bar(C::B_QE + qb), ((items >> 1) - 1) & 1, kWaitTimeoutNs)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(bar(C::B_QF + qb), x.n * C::kQ);
        for (int i = 0; i < x.n; ++i) {
          int h, row;
          walk.tile(p, x, i, h, row);
          for (int c = 0; c < C::KCH; ++c)
            tma_load_4d(s0 + C::off_q + (2 * qb + i) * C::kQ + c * kBM * 128, &tmQ,
                        bar(C::B_QF + qb), c * 64, row, h, x.b);
        }
        for (int t = 0; ok && t < x.steps; ++t) {
          load(&tmK, x, t, step_word(x, t, items, p.g.M));
          load(&tmV, x, t, 0);
        }
        ++items;
      }
      const int sl = slot_of();
      if (ok) {
        words[sl] = 0;
        mbar_arrive(bar(C::B_F + sl));
        ++g;
      }
      if (!ok) report_error(p.status, SPARGE_ERR_TIMEOUT);
      // Let the last loads land before the CTA can exit.
      for (int i = max(0, items - 2); i < items; ++i)
        mbar_wait(bar(C::B_QF + (i & 1)), (i >> 1) & 1, kWaitTimeoutNs);
      for (int i = max(0, g - C::NS); i < g; ++i)
        mbar_wait(bar(C::B_F + i % C::NS), (i / C::NS) & 1, kWaitTimeoutNs);
    }
    __syncwarp();
  } else if (warp >= kIssuer) {
    // ------------------------------------------------------------ products
    // A warp to a tile.  The whole warp runs the loop; one elected lane issues each MMA.
    constexpr uint32_t idS = idesc_bf16(kBM, kBN, false, false);
    constexpr uint32_t idO = idesc_bf16(kBM, D, false, true);
    const int i = warp - kIssuer;
    bool ok = true;
    int k = 0;              // steps so far: K(k) is tile 2 k of the ring, V(k) 2 k + 1
    int scored = 0, done = 0, begun = 0;  // of this tile: S, PV, items
    int items = 0;          // whose S was begun
    uint32_t zeroed = 0;    // parity of each slot's B_Z
    auto wait = [&](int b, int phase) {
      if (ok && !warp_wait(bar(b), phase & 1)) ok = false;
    };
    // S of the n-th step; returns its word.  Every slot and buffer is released by both
    // warps, by one without a tile too, and not before it was filled.
    auto score = [&](int n) -> int {
      const int sl = 2 * n % C::NS;
      wait(C::B_F + sl, 2 * n / C::NS);
      if (!ok) return 0;
      const int word = __shfl_sync(0xffffffffu, words[sl], 0);
      if (word == 0) return 0;
      const int qb = (word >> 4) & 1;
      if (word & 4) wait(C::B_QF + qb, items++ >> 1);
      if (!ok) return 0;
      if (i < (word & 3)) {
        tc_fence_after();
        const uint64_t dq = sdesc_sw128(s0 + C::off_q + (2 * qb + i) * C::kQ, 16, 1024);
        const uint64_t dk = sdesc_sw128(s0 + C::off_kv + sl * C::kKV, 16, 1024);
        const int buf = scored++ & 1;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          warp_mma_bf16(tmem + i * 128 + buf * kBN,
                        sdesc_add(dq, (kk >> 2) * (kBM * 128) + (kk & 3) * 32),
                        sdesc_add(dk, (kk >> 2) * (kBN * 128) + (kk & 3) * 32), idS, kk > 0);
        warp_commit(bar(C::B_S + 2 * i + buf));
      }
      warp_commit(bar(C::B_E + sl));
      if (word & 8) warp_commit(bar(C::B_QE + qb));
      return word;
    };
    // S runs two steps ahead of PV, which reads P in the place of S.
    int word = score(0), second = word != 0 ? score(1) : 0;
    for (; ok && word != 0; ++k) {
      const int sl = (2 * k + 1) % C::NS;
      wait(C::B_F + sl, (2 * k + 1) / C::NS);
      const int valid = word >> 8;
      if (i < (word & 3)) {
        // Keys behind the sample's length have P = 0, but their V may hold anything.
        if (ok && valid < kBN) {
          if (i == 0) {
            zero_tile_rows(sm + C::off_kv + sl * C::kKV, C::KCH, kBN * 128, valid, kBN, lane);
            if (lane == 0) mbar_arrive(bar(C::B_Z + sl));
          } else {
            wait(C::B_Z + sl, zeroed >> sl);
          }
        }
        if ((word & 4) != 0 && begun++ > 0) wait(C::B_OE + i, begun - 2);
        const int buf = done & 1;
        wait(C::B_P + 2 * i + buf, done++ >> 1);
        if (!ok) break;
        tc_fence_after();
        const uint64_t dv = sdesc_sw128(s0 + C::off_kv + sl * C::kKV, kBN * 128, 1024);
#pragma unroll
        for (int kk = 0; kk < kBN / 16; ++kk)
          warp_mma_bf16_ta(tmem + C::col_o + i * D, tmem + i * 128 + buf * kBN + kk * 8,
                           sdesc_add(dv, kk * 2048), idO, ((word & 4) == 0 || kk > 0) ? 1u : 0u);
        warp_commit(bar(C::B_PV + i));
        if (word & 8) warp_commit(bar(C::B_O + i));
      }
      if (!ok) break;
      if (valid < kBN) zeroed ^= 1u << sl;
      warp_commit(bar(C::B_E + sl));
      word = second;
      second = second != 0 ? score(k + 2) : 0;
    }
    if (!ok && lane == 0) report_error(p.status, SPARGE_ERR_TIMEOUT);
    warp_commit(bar(C::B_DONE));
    warp_wait(bar(C::B_DONE), 0);
  } else if (warp >= kOutput) {
    // ------------------------------------------------------------ output
    // A thread to a row, of one tile after the other.
    const int quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const float2* stats = reinterpret_cast<const float2*>(sm + C::off_row);
    bool ok = true;
    int items = 0, done[2] = {0, 0};
    Walk walk(p);
    for (Item x; ok && walk.next(p, x);) {
      const int qb = items & 1;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (i >= x.n) continue;
        int h, row0;
        walk.tile(p, x, i, h, row0);
        const bool in_range = row0 + r < p.g.N;
        float* lse = p.lse == nullptr
                         ? nullptr
                         : p.lse + (static_cast<int64_t>(x.b) * p.g.H + h) * p.g.N + row0 + r;
        if (x.steps == 0) {
          if (in_range) {
            __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.o.p) + x.b * p.o.sb +
                                  h * p.o.sh + static_cast<int64_t>(row0 + r) * p.o.sn;
            for (int c = 0; c < D; c += 8)
              *reinterpret_cast<uint4*>(orow + c) = make_uint4(0u, 0u, 0u, 0u);
            if (lse != nullptr) *lse = -INFINITY;
          }
          continue;
        }
        if (!warp_wait(bar(C::B_L + i), done[i] & 1) || !warp_wait(bar(C::B_O + i), done[i] & 1)) {
          ok = false;
          break;
        }
        ++done[i];
        tc_fence_after();
        const float2 ml = stats[i * kBM + r];
        const bool good = !(ml.y <= 0.f);  // (a sum that is NaN stays one)
        const float inv = good ? 1.f / ml.y : 0.f;
        // The output goes where the tile's queries were, and from there to memory.
        const uint32_t stage = C::off_q + (2 * qb + i) * C::kQ;
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += 32) {
          float f[32];
          tmem_ld32(lanes + C::col_o + i * D + c0, f);
          uint32_t w[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) w[c] = pack_bf16x2(f[2 * c] * inv, f[2 * c + 1] * inv);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint4*>(sm + stage + (c0 >> 6) * (kBM * 128) +
                                      sw128_offset(r, (c0 & 63) * 2 + 16 * c)) =
                make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        }
        tc_fence_before();
        mbar_arrive(bar(C::B_OE + i));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          for (int c = 0; c < C::KCH; ++c)
            tma_store_4d(&tmO, s0 + stage + c * (kBM * 128) + quarter * 32 * 128, c * 64,
                         row0 + quarter * 32, h, x.b);
          bulk_commit();
        }
        if (in_range && lse != nullptr) *lse = good ? (ml.x + log2f(ml.y)) * kLn2 : -INFINITY;
      }
      if (x.steps == 0) continue;
      ++items;
      if (ok && lane == 0) {
        bulk_wait_read();
        mbar_arrive(bar(C::B_QE + qb));
      }
      __syncwarp();
    }
    if (!ok) report_error(p.status, SPARGE_ERR_TIMEOUT);
    if (lane == 0) bulk_wait();  // every output is out
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    // A thread to a row of a tile.
    const int quarter = warp & 3, i = warp >> 2;
    const int r = quarter * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t oa = lanes + C::col_o + i * D;
    const uint64_t sl2 = f32x2(p.scale_log2, p.scale_log2);
    const float masked = p.scale_log2 > 0.f ? -INFINITY : INFINITY;
    bool ok = true;
    int steps = 0, items = 0;  // of this tile
    Walk walk(p);
    for (Item y; ok && walk.next(p, y);) {
      if (i >= y.n || y.steps == 0) continue;
      float m = 0.f, l = 0.f;
      for (int t = 0; t < y.steps; ++t, ++steps) {
        if (!warp_wait(bar(C::B_S + 2 * i + (steps & 1)), (steps >> 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sa = lanes + i * 128 + (steps & 1) * kBN;
        const int valid = y.len - t * kBN;
        if (t == 0) {
          // A first reference: the largest of 16 scores.
          uint32_t a[16];
          SPARGE_TMEM_LD_X16(sa, a);
          SPARGE_TMEM_WAIT_LD16(a);
          float top = -INFINITY;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (e < valid) top = fmaxf(top, __uint_as_float(a[e]) * p.scale_log2);
          m = top;
        }
        uint32_t pk[32];
        for (int pass = 0;; ++pass) {
          const bool none = m == -INFINITY;
          const float ref = none ? 0.f : m;
          const uint64_t nm2 = f32x2(-ref, -ref);
          uint64_t rs[2] = {f32x2(0.f, 0.f), f32x2(0.f, 0.f)};
          float top[2] = {-INFINITY, -INFINITY};
          uint32_t s[2][16];
          SPARGE_TMEM_LD_X16(sa, s[0]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t* a = s[c & 1];
            SPARGE_TMEM_WAIT_LD16(a);
            if (c < 3) SPARGE_TMEM_LD_X16(sa + 16 * c + 16, s[(c + 1) & 1]);  // comes in meanwhile
            if (valid < 16 * c + 16) {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (16 * c + e >= valid) a[e] = __float_as_uint(masked);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint64_t v = ffma2(f32x2(__uint_as_float(a[2 * e]), __uint_as_float(a[2 * e + 1])),
                                       sl2, nm2);
              const float v0 = f32x2_lo(v), v1 = f32x2_hi(v);
              top[e & 1] = fmax3(top[e & 1], v0, v1);
              const float p0 = ex2_approx(v0), p1 = ex2_approx(v1);
              rs[e & 1] = fadd2(rs[e & 1], f32x2(p0, p1));
              pk[8 * c + e] = pack_bf16x2(p0, p1);
            }
          }
          const float over = fmaxf(top[0], top[1]);
          // Decided for the whole warp: tensor memory is read and written by warps.  One
          // repetition is enough, and all there is: scores past 2^30 or so could not move
          // the reference by their distance to it.
          const bool move = over > (none ? -INFINITY : kSlack);
          if (pass > 0 || !__any_sync(0xffffffffu, move)) {
            const uint64_t sum = fadd2(rs[0], rs[1]);
            l += f32x2_lo(sum) + f32x2_hi(sum);
            break;
          }
          const float up = move ? over : 0.f;
          const float alpha = none ? 1.f : exp2f(-up);  // (1 for a sum and an output of 0)
          if (move) m = ref + up;
          l *= alpha;
          if (t > 0) {
            // O holds the steps before this one once the last of them is done.  (S of
            // this step being there, the one before that is.)
            if (!warp_wait(bar(C::B_PV + i), (steps - 1) & 1)) ok = false;
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 16) {
              uint32_t ro[16];
              SPARGE_TMEM_LD_X16(oa + c0, ro);
              SPARGE_TMEM_WAIT_LD16(ro);
#pragma unroll
              for (int c = 0; c < 16; ++c) ro[c] = __float_as_uint(__uint_as_float(ro[c]) * alpha);
              SPARGE_TMEM_ST_X16(oa + c0, ro);
            }
            tmem_st_wait();
          }
        }
        // P over the first 32 of the 64 columns of S.
        SPARGE_TMEM_ST_X16(sa, pk);
        SPARGE_TMEM_ST_X16(sa + 16, (pk + 16));
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar(C::B_P + 2 * i + (steps & 1)));
      }
      // The last item's must have been read.
      if (ok && items > 0 && !warp_wait(bar(C::B_OE + i), (items - 1) & 1)) ok = false;
      if (!ok) break;
      ++items;
      reinterpret_cast<float2*>(sm + C::off_row)[i * kBM + r] = make_float2(m, l);
      mbar_arrive(bar(C::B_L + i));
    }
    if (!ok) report_error(p.status, SPARGE_ERR_TIMEOUT);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch_wide(const CrossGeom& g, const sparge_cross& a, cudaStream_t st) {
  using C = WideCfg<D>;
  CUtensorMap tq, tk, tv, to;
  if (make_tmap_bf16_4d(&to, a.o, g.B, g.H, g.N, D, a.o_stride, 32) != 0 ||
      make_tmap_bf16_4d(&tq, a.q, g.B, g.H, g.N, D, a.q_stride, kBM) != 0 ||
      make_tmap_bf16_4d(&tk, a.k, g.Bk, g.Hk, g.M, D, a.k_stride, kBN) != 0 ||
      make_tmap_bf16_4d(&tv, a.v, g.Bk, g.Hk, g.M, D, a.v_stride, kBN) != 0)
    return cudaErrorInvalidValue;
  WideParams p = {};
  p.g = g;
  p.o = {a.o, a.o_stride[0], a.o_stride[1], a.o_stride[2]};
  p.lse = a.lse;
  p.scale_log2 = g.scale * kLog2e;
  p.even = (g.group * g.Mq + 1) / 2 * 2;
  p.tiles = g.B * g.Hk * p.even;
  p.spread = g.kv_len != nullptr;
  p.status = a.status;
  const cudaError_t e = cudaFuncSetAttribute(
      cross_fwd_wide_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::bytes);
  if (e != cudaSuccess) return e;
  const int grid = std::min(p.tiles / 2, kSMs);
  cross_fwd_wide_kernel<D><<<grid, kThreads, C::bytes, st>>>(tq, tk, tv, to, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cross_fwd_wide(const CrossGeom& g, const sparge_cross& a, cudaStream_t st) {
  return g.d == 128 ? launch_wide<128>(g, a, st) : launch_wide<64>(g, a, st);
}

}  // namespace sparge
