// Row slots: what the row kernels around the attention share (the head
// layout kernels and the residual norm kernels).
//
// A slot is a group of W warps that owns one row (token) of C channels at a
// time, eight consecutive channels to a thread, so per-channel operands
// (weights, gates, scales) and per-channel sums stay in its registers from row
// to row.  A slot takes T rows at once: their loads are all in flight together
// and one barrier serves the sums of all T.  Slots of one CTA are independent
// of one another: each has its own named barrier, or none when W is 1.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace sparge {

constexpr int kSMs = 152;              // of a GB300: sizes grids and workspaces
constexpr int kMaxRowChannels = 8192;  // 32 warps of 8 channels a thread
constexpr int kMaxSlots = 8;           // per CTA; named barriers 1 .. 8

// Warps of one slot, and slots of one CTA: enough to make 8 warps of a CTA
// where a row needs fewer.
__host__ __device__ inline int slot_warps(int C) { return (C + 255) / 256; }
__host__ __device__ inline int slots_per_cta(int W) { return W >= kMaxSlots ? 1 : kMaxSlots / W; }

// A kernel is built for three sizes of CTA (threads, rows a slot takes at
// once): the registers of a thread shrink as rows get wider.
struct Tier {
  int threads, fwd_rows, bwd_rows;
};
constexpr Tier kTiers[3] = {{256, 4, 2}, {640, 2, 1}, {1024, 1, 1}};
inline int tier_of(int threads) {
  return threads <= kTiers[0].threads ? 0 : threads <= kTiers[1].threads ? 1 : 2;
}

struct Slot {
  int index;    // in the CTA
  int W, warp;  // warps of the slot; this thread's among them
  int lane, tid;
  float* red;   // 2 * W * kSlotRed floats of shared memory
  int phase;
};

// Floats one warp contributes to a slot reduction, at most.
constexpr int kSlotRed = 8;
constexpr int kSlotRedFloats = 2 * 32 * kSlotRed;  // of a CTA of at most 32 warps

SPARGE_DEV Slot make_slot(int W, float* red) {
  Slot s;
  const int warp = threadIdx.x >> 5;
  s.lane = threadIdx.x & 31;
  s.index = warp / W;
  s.W = W;
  s.warp = warp - s.index * W;
  s.tid = s.warp * 32 + s.lane;
  s.red = red + s.index * W * 2 * kSlotRed;
  s.phase = 0;
  return s;
}

SPARGE_DEV void slot_sync(const Slot& s) {
  if (s.W == 1)
    __syncwarp();
  else
    named_barrier_sync(1 + s.index, s.W * 32);
}

// Sums v[0..K) over the slot's threads; every thread gets the sums.  The two
// halves of `red` alternate, so one barrier a call is enough: a warp cannot
// reach the next but one call before every warp has read this one's sums.
template <int K>
SPARGE_DEV void slot_sum(Slot& s, float (&v)[K]) {
  static_assert(K <= kSlotRed, "reduction buffer");
#pragma unroll
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  }
  if (s.W == 1) return;
  float* red = s.red + s.phase * s.W * kSlotRed;
  s.phase ^= 1;
  if (s.lane == 0) {
#pragma unroll
    for (int k = 0; k < K; ++k) red[s.warp * kSlotRed + k] = v[k];
  }
  slot_sync(s);
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = 0.f;
  for (int w = 0; w < s.W; ++w) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += red[w * kSlotRed + k];
  }
}

// ------------------------------------------------- eight values of a thread
template <typename T>
struct Raw8;  // eight values as loaded
template <>
struct Raw8<__nv_bfloat16> {
  uint4 v[1];
};
template <>
struct Raw8<float> {
  uint4 v[2];
};

SPARGE_DEV uint2 ldg8_no_l1(const void* ptr) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "l"(ptr));
  return v;
}

// Eight consecutive values (16-byte aligned), read once.
template <typename T>
SPARGE_DEV Raw8<T> load8(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
    r.v[i] = ldg_no_l1(reinterpret_cast<const uint4*>(p) + i);
  return r;
}

// Four values at p and four at q.
SPARGE_DEV Raw8<__nv_bfloat16> load4x2(const __nv_bfloat16* p, const __nv_bfloat16* q) {
  const uint2 a = ldg8_no_l1(p), b = ldg8_no_l1(q);
  return {{make_uint4(a.x, a.y, b.x, b.y)}};
}
SPARGE_DEV Raw8<float> load4x2(const float* p, const float* q) {
  return {{ldg_no_l1(reinterpret_cast<const uint4*>(p)),
           ldg_no_l1(reinterpret_cast<const uint4*>(q))}};
}

template <typename T>
SPARGE_DEV Raw8<T> zero8() {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) r.v[i] = make_uint4(0, 0, 0, 0);
  return r;
}

SPARGE_DEV void unpack8(const Raw8<__nv_bfloat16>& r, float (&f)[8]) {
  const uint32_t u[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
SPARGE_DEV void unpack8(const Raw8<float>& r, float (&f)[8]) {
  const uint32_t u[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w,
                         r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(u[i]);
}

SPARGE_DEV Raw8<__nv_bfloat16> pack8(const float (&f)[8], __nv_bfloat16) {
  return {{make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]))}};
}
SPARGE_DEV Raw8<float> pack8(const float (&f)[8], float) {
  return {{make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3])),
           make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]),
                      __float_as_uint(f[7]))}};
}

template <typename T>
SPARGE_DEV void store8(T* p, const float (&f)[8]) {
  const Raw8<T> r = pack8(f, T());
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = r.v[i];
}
SPARGE_DEV void store4x2(__nv_bfloat16* p, __nv_bfloat16* q, const float (&f)[8]) {
  const Raw8<__nv_bfloat16> r = pack8(f, __nv_bfloat16());
  *reinterpret_cast<uint2*>(p) = make_uint2(r.v[0].x, r.v[0].y);
  *reinterpret_cast<uint2*>(q) = make_uint2(r.v[0].z, r.v[0].w);
}
SPARGE_DEV void store4x2(float* p, float* q, const float (&f)[8]) {
  const Raw8<float> r = pack8(f, 0.f);
  *reinterpret_cast<uint4*>(p) = r.v[0];
  *reinterpret_cast<uint4*>(q) = r.v[1];
}

// ------------------------------------------------------- sums of partial rows
// out[o][c] = sum over r < nrow, in that order, of src[(o * nrow + r) * ld + c].
struct ReduceJob {
  const float* src;
  void* out;
  int64_t ld;
  int nrow, nout, C;
  int out_bf16;
};
constexpr int kReduceJobs = 4;
struct ReduceJobs {
  ReduceJob job[kReduceJobs];
  int n;
};

// Launches the sums on `st` behind the kernel that writes the partial rows
// (programmatic dependent launch).
cudaError_t launch_reduce_rows(const ReduceJobs& jobs, cudaStream_t st);

// Lets the next kernel of the stream start; waits for the one before.
SPARGE_DEV void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
SPARGE_DEV void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace sparge
