// Sums of the partial rows that the row kernels leave (one row of per-channel
// sums a slot), in a fixed order: repeated calls give the same bits.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "rows.cuh"

namespace sparge {

namespace {

// A warp sums 128 channels (four to a lane) of some of an output's partial
// rows, eight loads in flight.  With many rows to a sum the 32 warps of a CTA
// take a slice each and add the slices in order; with few every warp has a sum
// of its own (a modulation for each of 21 frames, 14 rows each: 3 us instead of
// 13 with 32 slices of half a row).
constexpr int kWarps = 32;
constexpr int kFewRows = 32;

SPARGE_DEV void add4(float4& a, const float4& b) { a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w; }

SPARGE_DEV void put4(const ReduceJob& j, int64_t at, const float4& v) {
  if (j.out_bf16)
    reinterpret_cast<uint2*>(j.out)[at / 4] = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  else
    reinterpret_cast<float4*>(j.out)[at / 4] = v;
}

__global__ void __launch_bounds__(32 * kWarps) reduce_rows_kernel(
    const __grid_constant__ ReduceJobs jobs) {
  __shared__ float4 part[kWarps][32];
  grid_wait();
  const ReduceJob& j = jobs.job[blockIdx.y];
  const int chunks = (j.C + 127) / 128, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool few = j.nrow <= kFewRows;
  const int64_t item = few ? static_cast<int64_t>(blockIdx.x) * kWarps + warp : blockIdx.x;
  const bool there = item < static_cast<int64_t>(chunks) * j.nout;
  const int o = there ? static_cast<int>(item / chunks) : 0;
  const int c = (static_cast<int>(item) - o * chunks) * 128 + lane * 4;
  const bool mine = there && c < j.C;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  if (mine) {
    const float* src = j.src + static_cast<int64_t>(o) * j.nrow * j.ld + c;
    const int step = few ? 1 : kWarps;
    int r = few ? 0 : warp;
    for (; r + 7 * step < j.nrow; r += 8 * step) {
      float4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = *reinterpret_cast<const float4*>(src + static_cast<int64_t>(r + i * step) * j.ld);
#pragma unroll
      for (int i = 0; i < 8; ++i) add4(sum, v[i]);
    }
    for (; r < j.nrow; r += step)
      add4(sum, *reinterpret_cast<const float4*>(src + static_cast<int64_t>(r) * j.ld));
  }
  if (few) {
    if (mine) put4(j, static_cast<int64_t>(o) * j.C + c, sum);
    return;
  }
  part[warp][lane] = sum;
  __syncthreads();
  // Halve the slices five times, always in the same order.
  for (int n = kWarps / 2; n > 0; n /= 2) {
    if (warp < n) {
      add4(sum, part[warp + n][lane]);
      part[warp][lane] = sum;
    }
    __syncthreads();
  }
  if (warp == 0 && mine) put4(j, static_cast<int64_t>(o) * j.C + c, sum);
}

}  // namespace

cudaError_t launch_reduce_rows(const ReduceJobs& jobs, cudaStream_t st) {
  int64_t most = 0;
  for (int i = 0; i < jobs.n; ++i) {
    const ReduceJob& j = jobs.job[i];
    const int64_t items = static_cast<int64_t>((j.C + 127) / 128) * j.nout;
    const int64_t n = j.nrow <= kFewRows ? (items + kWarps - 1) / kWarps : items;
    if (n > most) most = n;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(most), jobs.n);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, reduce_rows_kernel, jobs);
}

}  // namespace sparge
