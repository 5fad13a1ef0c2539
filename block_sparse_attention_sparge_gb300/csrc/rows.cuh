// Row slots: what the row kernels around the attention share (the head
// layout kernels and the residual norm kernels).
//
// A slot is a group of W warps that owns one row (token) of C channels at a
// time, V times eight channels to a thread, so per-channel
// operands (weights, gates, scales) and per-channel sums stay with the thread
// from row to row.  A slot takes T rows at once: one barrier serves the sums of
// all T.  Slots of one CTA are independent of one another: each has its own
// named barrier, or none when W is 1.
//
// Rows come in through a ring of shared-memory stages that every thread fills
// for itself (cp.async of its own channels) and alone reads: bytes stay in
// flight while earlier rows are computed, without registers to hold them and
// without a barrier.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace sparge {

constexpr int kSMs = 152;              // of a GB300: sizes grids and workspaces
constexpr int kSmemPerSm = 228 * 1024;  // shared memory of an SM
constexpr int kSmemOfCta = 1024;      // of it reserved for each CTA
constexpr int kSmemPerCta = 227 * 1024;  // that one CTA can ask for
constexpr int kMaxRowChannels = 8192;

constexpr int kMaxSlots = 6;            // per CTA; named barriers 1 .. 6

// A thread holds V times eight channels: one up to 1536 channels (CTAs of at most
// 192 threads), two above (512), so that wide rows too keep CTAs of few warps,
// several on an SM.
inline int row_vectors(int C) { return C <= 1536 ? 1 : 2; }
constexpr int row_threads(int V) { return V == 1 ? 192 : 512; }
// The backward, whose sums stay in registers, has no room for sixteen channels
// up to 5120 of them: there it takes eight and CTAs of up to 640 threads.  (One CTA
// an SM from 2816 channels on: of the copy rate, head layout and residual norm in
// bf16, 91 and 69 % at 2560, 68 and 72 at 2816, 77 and 81 at 4096, 82 and 85 at
// 5120; with sixteen channels 44 and 54 at 5376, 57 and 60 at 8192.)
inline int bwd_threads(int C) { return C <= 1536 ? 192 : C <= 5120 ? 640 : 512; }
constexpr int bwd_vectors(int threads) { return threads == 512 ? 2 : 1; }
// Eights of warps of a slot, of a kernel built for CTAs of so many threads.
constexpr int warp_eights(int threads) { return (threads / 32 + 7) / 8; }
// Registers of a thread that its CTAs leave: two of six warps an SM, one of
// twenty, one of sixteen.
constexpr int bwd_regs(int threads) { return threads == 192 ? 168 : threads == 640 ? 96 : 128; }
// Warps of one slot, and slots of one CTA: enough to make 6 warps of a CTA
// where a row needs fewer.
__host__ __device__ inline int slot_warps(int C, int V) { return (C + 256 * V - 1) / (256 * V); }
__host__ __device__ inline int slots_per_cta(int W) { return W >= kMaxSlots ? 1 : kMaxSlots / W; }

// Warps of `regs` registers a thread that an SM holds: each of its four
// schedulers has 512 registers a lane.
constexpr int resident_warps(int regs) { return 4 * (512 / regs); }

struct Slot {
  int index;    // in the CTA
  int W, warp;  // warps of the slot; this thread's among them
  int lane, tid;
  float* red;   // two halves of `half` floats of shared memory, zeros at the start
  int half;
  int phase;
};

// Floats a warp contributes to a slot's reduction, at most, in most kernels; of
// one half of a slot's buffer, in a kernel built for so many threads; and of the
// buffers of a CTA.
constexpr int kSlotRed = 4;
constexpr int red_half(int threads, int per_warp = kSlotRed) {
  return warp_eights(threads) * 8 * per_warp;
}
constexpr int red_floats(int threads, int per_warp = kSlotRed) {
  return kMaxSlots * 2 * red_half(threads, per_warp);
}

// Clears `red` (the CTA's buffers); a barrier of the CTA has to follow.
SPARGE_DEV Slot make_slot(int W, float* red, int half) {
  Slot s;
  // The shuffle tells the compiler that the warp's index is the same in all
  // lanes, so what follows from it is computed once for the warp.
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);
  s.lane = threadIdx.x & 31;
  s.index = warp / W;
  s.W = W;
  s.warp = warp - s.index * W;
  s.tid = s.warp * 32 + s.lane;
  s.red = red + s.index * 2 * half;
  s.half = half;
  for (int i = threadIdx.x; i < kMaxSlots * 2 * half; i += blockDim.x) red[i] = 0.f;
  s.phase = 0;
  return s;
}

SPARGE_DEV void slot_sync(const Slot& s) {
  if (s.W == 1)
    __syncwarp();
  else
    named_barrier_sync(1 + s.index, s.W * 32);
}

// Sums v[0..K) over the warp, K a power of two: each step halves the values a
// lane carries while it doubles the lanes behind each, so K sums take K + 4 or
// so shuffles instead of 5 K.  The sum of v[k] ends in the lanes l with
// l / (32 / K) == k.
template <int K>
SPARGE_DEV float warp_sums(const float (&in)[K], int lane) {
  static_assert(K == 1 || K == 2 || K == 4 || K == 8, "power of two");
  float v[K];
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = in[k];
  int o = 16;
#pragma unroll
  for (int m = K / 2; m >= 1; m /= 2, o /= 2) {
    const bool upper = lane & o;
#pragma unroll
    for (int k = 0; k < m; ++k) {
      const float keep = upper ? v[m + k] : v[k], send = upper ? v[k] : v[m + k];
      v[k] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
#pragma unroll
  for (; o > 0; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  return v[0];
}

// Joins the warps of a slot.  Every warp leaves up to four floats (eight in the
// head layout's backward of two tokens) in its row of `red`; every warp then reads
// all of them at once, lane l the float l / 8 (or the two from l / 8 * 2) of warps
// l % 8, l % 8 + 8 and so on, and finishes with three shuffles instead of a loop
// over the warps.  The two halves of `red`
// alternate, so one barrier a call is enough: a warp cannot reach the next but
// one call before every warp has read this one's values.
SPARGE_DEV float* slot_half(Slot& s) {
  float* red = s.red + s.phase * s.half;
  s.phase ^= 1;
  return red;
}
// Sum over the eight lanes of a group.
SPARGE_DEV float sum_of_8(float v) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums v[0..K) over the slot's threads; every thread gets the sums.  A slot of
// the kernel has at most 8 * EIGHTS warps.
template <int EIGHTS, int K>
SPARGE_DEV void slot_sum(Slot& s, float (&v)[K]) {
  const float mine = warp_sums(v, s.lane);
  if (s.W == 1) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = __shfl_sync(0xffffffffu, mine, k * (32 / K));
    return;
  }
  constexpr int R = K > kSlotRed ? K : kSlotRed;  // floats of a warp
  float* red = slot_half(s);
  if (s.lane % (32 / K) == 0) red[s.warp * R + s.lane / (32 / K)] = mine;
  slot_sync(s);
  if constexpr (K <= 4) {
    const float* in = red + (s.lane & 7) * R + (s.lane >> 3) % K;
    float sum = in[0];
#pragma unroll
    for (int e = 1; e < EIGHTS; ++e) sum += in[8 * e * R];
    sum = sum_of_8(sum);
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = __shfl_sync(0xffffffffu, sum, 8 * k);
  } else {
    static_assert(K == 8, "two floats of a warp to a lane");
    const float2* in = reinterpret_cast<const float2*>(red + (s.lane & 7) * R) + (s.lane >> 3);
    float2 sum = in[0];
#pragma unroll
    for (int e = 1; e < EIGHTS; ++e) {
      const float2 more = in[8 * e * R / 2];
      sum.x += more.x, sum.y += more.y;
    }
    sum.x = sum_of_8(sum.x);
    sum.y = sum_of_8(sum.y);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __shfl_sync(0xffffffffu, sum.x, 8 * k);
      v[2 * k + 1] = __shfl_sync(0xffffffffu, sum.y, 8 * k);
    }
  }
}

// ------------------------------------------------------ stages of a thread
SPARGE_DEV void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
SPARGE_DEV void cp_async8(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
SPARGE_DEV void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
SPARGE_DEV void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// A thread's pieces of 16 bytes, `pitch` (the threads of the CTA) apart, so the
// pieces that a warp copies lie side by side.  (Laid out thread by thread
// instead, a copy of two bf16 tensors into a third runs at 4.1 TB/s, not 6.3.)
struct Ring {
  uint4* p;
  int pitch;
  SPARGE_DEV Ring operator+(int k) const { return {p + k * pitch, pitch}; }
  SPARGE_DEV uint4& operator[](int k) const { return p[k * pitch]; }
};
template <typename T>
constexpr int pieces8() {  // pieces of eight values
  return static_cast<int>(sizeof(T)) / 2;
}

// Launches a kernel with `smem` bytes of dynamic shared memory.  `most` is what
// any call of this kernel can ask for: the limit belongs to the kernel on its
// device, not to the call, so set to a call's own size it could be lowered by
// another host thread between the setting and the launch, which then fails.
template <typename Kernel, typename Params>
cudaError_t launch_row_kernel(Kernel* kernel, const Params& p, dim3 grid, int threads, int smem,
                              int most, cudaStream_t st) {
  if (most > 42 * 1024) {  // 48 KB less what the kernels declare
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) {
      cudaGetLastError();  // the next launch must not report it
      return e;
    }
  }
  kernel<<<grid, threads, smem, st>>>(p);
  return cudaGetLastError();
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

// Eight consecutive values (16-byte aligned), read once.
template <typename T>
SPARGE_DEV Raw8<T> load8(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < pieces8<T>(); ++i) r.v[i] = ldg_no_l1(reinterpret_cast<const uint4*>(p) + i);
  return r;
}

template <typename T>
SPARGE_DEV Raw8<T> zero8() {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < pieces8<T>(); ++i) r.v[i] = make_uint4(0, 0, 0, 0);
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
SPARGE_DEV void store_raw8(T* p, const Raw8<T>& r) {
#pragma unroll
  for (int i = 0; i < pieces8<T>(); ++i) reinterpret_cast<uint4*>(p)[i] = r.v[i];
}
template <typename T>
SPARGE_DEV void store8(T* p, const float (&f)[8]) {
  store_raw8(p, pack8(f, T()));
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

// Eight values into the ring at dst, and back out: in a row at p, or four at p
// and four at q.
template <typename T>
SPARGE_DEV void stage8(Ring dst, const T* p) {
#pragma unroll
  for (int i = 0; i < pieces8<T>(); ++i) cp_async16(&dst[i], reinterpret_cast<const uint4*>(p) + i);
}
SPARGE_DEV void stage4x2(Ring dst, const __nv_bfloat16* p, const __nv_bfloat16* q) {
  cp_async8(&dst[0], p);
  cp_async8(reinterpret_cast<uint2*>(&dst[0]) + 1, q);
}
SPARGE_DEV void stage4x2(Ring dst, const float* p, const float* q) {
  cp_async16(&dst[0], p);
  cp_async16(&dst[1], q);
}
template <typename T>
SPARGE_DEV Raw8<T> unstage8(Ring src) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < pieces8<T>(); ++i) r.v[i] = src[i];
  return r;
}

// ------------------------------------------------------- sums of partial rows
// out[o][c] = sum over r < nrow of src[(o * nrow + r) * ld + c], in an order that
// depends on nrow alone.  C and ld are multiples of 4, nout * C is below 2^31;
// 16-byte aligned (out: 8 for bf16).
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
