// Sums of the partial rows that the row kernels leave (one row of per-channel
// sums a CTA of the head layout, a slot or a share of a group of the residual
// norm), in a fixed order: repeated calls give the same bits.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "rows.cuh"

namespace sparge {

namespace {

// A warp sums 128 channels (four to a lane) of a slice of an output's partial
// rows, eight loads in flight.  A sum has as many slices, neighbouring warps of a
// CTA, as leave each some eight rows, and adds them in order.  Bound by latency:
// 24 rows of 128 take 3 us behind the kernel that leaves them (10 with a single
// warp a sum).  The stated minimum of one CTA keeps the loads together: without
// it the compiler holds to 32 registers and waits for them one by one (2.5 us
// more in every backward).
constexpr int kWarps = 32;

__host__ __device__ inline int slices_of(int nrow) {
  int n = 1;
  while (n < kWarps && n * 8 < nrow) n *= 2;
  return n;
}

SPARGE_DEV void add4(float4& a, const float4& b) { a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w; }

SPARGE_DEV void put4(const ReduceJob& j, int64_t at, const float4& v) {
  if (j.out_bf16)
    reinterpret_cast<uint2*>(j.out)[at / 4] = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  else
    reinterpret_cast<float4*>(j.out)[at / 4] = v;
}

__global__ void __launch_bounds__(32 * kWarps, 1) reduce_rows_kernel(
    const __grid_constant__ ReduceJobs jobs) {
  __shared__ float4 part[kWarps][32];
  grid_wait();
  const ReduceJob& j = jobs.job[blockIdx.y];
  const int chunks = (j.C + 127) / 128, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int slices = slices_of(j.nrow), slice = warp & (slices - 1);
  const int item = blockIdx.x * (kWarps / slices) + warp / slices;
  const bool there = item < chunks * j.nout;
  const int o = there ? item / chunks : 0;
  const int c = (item - o * chunks) * 128 + lane * 4;
  const bool mine = there && c < j.C;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  if (mine) {
    const float* src = j.src + static_cast<int64_t>(o) * j.nrow * j.ld + c;
    for (int r = slice; r < j.nrow; r += 8 * slices) {
      // (Clamped, not skipped: a branch around each load would wait for it.)
      float4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = *reinterpret_cast<const float4*>(
            src + static_cast<int64_t>(min(r + i * slices, j.nrow - 1)) * j.ld);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (r + i * slices < j.nrow) add4(sum, v[i]);
    }
  }
  if (slices > 1) {
    part[warp][lane] = sum;
    __syncthreads();
    if (slice > 0) return;
#pragma unroll 8
    for (int i = 1; i < slices; ++i) add4(sum, part[warp + i][lane]);
  }
  if (mine) put4(j, static_cast<int64_t>(o) * j.C + c, sum);
}

}  // namespace

cudaError_t launch_reduce_rows(const ReduceJobs& jobs, cudaStream_t st) {
  int64_t most = 0;
  for (int i = 0; i < jobs.n; ++i) {
    const ReduceJob& j = jobs.job[i];
    const int64_t items = static_cast<int64_t>((j.C + 127) / 128) * j.nout;
    const int per_cta = kWarps / slices_of(j.nrow);
    const int64_t n = (items + per_cta - 1) / per_cta;
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
