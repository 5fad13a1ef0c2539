// Sums of the partial rows that the row kernels leave (one row of per-channel
// sums a slot), in a fixed order: repeated calls give the same bits.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "rows.cuh"

namespace sparge {

namespace {

// A CTA sums 32 channels: 32 slices of the rows, eight loads of a thread in
// flight, then the slices in order.
constexpr int kSlices = 32;

__global__ void __launch_bounds__(32 * kSlices) reduce_rows_kernel(
    const __grid_constant__ ReduceJobs jobs) {
  __shared__ float part[kSlices][33];
  grid_wait();
  const ReduceJob& j = jobs.job[blockIdx.y];
  const int chunks = (j.C + 31) / 32;
  if (blockIdx.x >= static_cast<unsigned>(chunks * j.nout)) return;
  const int o = blockIdx.x / chunks, lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int c = (blockIdx.x - o * chunks) * 32 + lane;
  float sum = 0.f;
  if (c < j.C) {
    const float* src = j.src + static_cast<int64_t>(o) * j.nrow * j.ld + c;
    int r = slice;
    for (; r + 7 * kSlices < j.nrow; r += 8 * kSlices) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = src[static_cast<int64_t>(r + i * kSlices) * j.ld];
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += v[i];
    }
    for (; r < j.nrow; r += kSlices) sum += src[static_cast<int64_t>(r) * j.ld];
  }
  part[slice][lane] = sum;
  __syncthreads();
  // Warp s adds the slices of channel s: slice index in the lane.
  float v = part[lane][slice];
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
  const int oc = (blockIdx.x - o * chunks) * 32 + slice;
  if (lane == 0 && oc < j.C) {
    const int64_t at = static_cast<int64_t>(o) * j.C + oc;
    if (j.out_bf16)
      static_cast<__nv_bfloat16*>(j.out)[at] = __float2bfloat16_rn(v);
    else
      static_cast<float*>(j.out)[at] = v;
  }
}

}  // namespace

cudaError_t launch_reduce_rows(const ReduceJobs& jobs, cudaStream_t st) {
  unsigned most = 0;
  for (int i = 0; i < jobs.n; ++i) {
    const unsigned n = static_cast<unsigned>((jobs.job[i].C + 31) / 32) * jobs.job[i].nout;
    if (n > most) most = n;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(most, jobs.n);
  cfg.blockDim = dim3(32 * kSlices);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, reduce_rows_kernel, jobs);
}

}  // namespace sparge
