// Global norm of a list of gradient tensors, and the gradients scaled to it.
//
//   norm = sqrt(sum over all tensors of g^2)
//   c    = min(1, max_norm / (norm + eps));   out = g * c
//
// Two launches: every CTA of the first leaves its sum of squares (fp64) in the
// workspace; every CTA of the second adds those in the same fixed order, so all
// get the same bits, and scales its chunks.  The second takes the chunks in
// reverse: the ones that the first read last are still in L2.
//
// A thread squares and adds 64 values in fp32, four such sums at a time, then
// adds that to an fp64 sum.  Where a sum left the range in which no square that
// matters over- or underflows (below 2^-90 or above 2^124), its values are read
// again and scaled by a power of two first, so gradients of any size that fp32
// holds give a norm of full precision.  fp64 runs at 1/60 of the fp32 rate here
// (an addition of a warp takes the pipe some 15 cycles): one for every 32 values
// kept the pipe busy half of the time, and the last sums are left to single
// warps (a list of four small tensors: 6 us, 13 with all threads at it).
//
// Bound by memory: 680M bf16 values take 203 us for the norm (6.7 TB/s) and 593
// us in all, which is three passes over 1.36 GB at the rate of a copy; the second
// read is the price of a factor that only the whole norm gives.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <new>

#include "common.cuh"
#include "rows.cuh"
#include "sparge.h"

namespace sparge {

namespace {

constexpr int kClipThreads = 256;
// Vectors of eight values that a thread takes at a time: eight keep the memory
// busy; lists that would not give every SM a chunk of that size take one (four
// tensors of 16384 values: 5 us, 8 with eight).
constexpr int kFewVectors = 1, kVectors = 8;
constexpr int chunk_values(int vectors) { return kClipThreads * 8 * vectors; }
// The first launch is resident as a whole; the second runs in waves, whose CTAs
// end one by one instead of all with the slowest (634 us in one, 603 in five,
// 599 in eleven).
constexpr int kNormCtas = kSMs * 3, kScaleCtas = kSMs * 32;
constexpr int kSmallList = 48, kLargeList = 1024;  // tensors of one launch

// A list of tensors as a kernel parameter (29704 of the 32764 bytes there are for
// the large one; a launch copies all of it, so short lists have a small one).
template <int MAX>
struct ClipList {
  const void* in[MAX];
  void* out[MAX];
  int64_t numel[MAX];
  uint32_t chunk[MAX + 1];  // first chunk of each tensor
  uint8_t bf16[MAX];
  int n;
};

struct ClipArgs {
  double* sums;  // [all CTAs of the first launches]
  int n_sums;
  float* norm;  // written by the first CTA of the launch that has it
  float max_norm, eps;
  int in_place;
};

static_assert(sizeof(ClipList<kLargeList>) + sizeof(ClipArgs) <= 32764, "kernel parameters");

// A chunk: values [base, base + left) of tensor i, or the first of them.
struct Chunk {
  int i;
  int64_t base, left;
};

// Finds chunk c by bisection of the chunk starts, among tensors [lo, hi).
template <int VEC, int MAX>
SPARGE_DEV Chunk find(const ClipList<MAX>& l, uint32_t c, int lo, int hi) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (l.chunk[mid] <= c) lo = mid;
    else hi = mid;
  }
  const int64_t base = static_cast<int64_t>(c - l.chunk[lo]) * chunk_values(VEC);
  return {lo, base, l.numel[lo] - base};
}

// The place in a chunk of this thread's k-th group of eight values.
SPARGE_DEV int place(int k) { return (k * kClipThreads + static_cast<int>(threadIdx.x)) * 8; }

// Sum of the squares of eight values.
SPARGE_DEV void square8(const float (&f)[8], uint64_t& a, uint64_t& b) {
  const uint64_t p = f32x2(f[0], f[1]), q = f32x2(f[2], f[3]);
  const uint64_t r = f32x2(f[4], f[5]), s = f32x2(f[6], f[7]);
  a = ffma2(p, p, a);
  b = ffma2(q, q, b);
  a = ffma2(r, r, a);
  b = ffma2(s, s, b);
}

// A thread's sum: four chunks' worth in fp32, then on to fp64.
struct Sum {
  double total = 0.0;
  float part = 0.f;
  int n = 0;
  SPARGE_DEV void add(float s) {
    part += s;
    if (++n == 4) flush();
  }
  SPARGE_DEV void flush() {
    total += part;
    part = 0.f;
    n = 0;
  }
};

// Sum of the squares of this thread's values of a chunk, scaled by f before they
// are squared (SCALED).  `ahead` runs while the loads are in flight.
template <int VEC, bool SCALED, typename T, typename Ahead>
SPARGE_DEV float chunk_squares(const T* in, int64_t left, float f, const Ahead& ahead) {
  uint64_t a = 0, b = 0;
  if ((reinterpret_cast<uintptr_t>(in) & 15) == 0) {
    Raw8<T> r[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const int at = place(k);
      r[k] = at + 8 <= left ? load8(in + at) : zero8<T>();
    }
    ahead();
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      float v[8];
      unpack8(r[k], v);
      if (SCALED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= f;
      }
      square8(v, a, b);
    }
    // The last values of a tensor whose size is no multiple of eight.
    const int64_t whole = left & ~int64_t(7);
    if (left < chunk_values(VEC) && threadIdx.x < left - whole) {
      const float v = SCALED ? static_cast<float>(in[whole + threadIdx.x]) * f
                             : static_cast<float>(in[whole + threadIdx.x]);
      a = ffma2(f32x2(v, 0.f), f32x2(v, 0.f), a);
    }
  } else {
    // Off a 16-byte boundary a value at a time (170M bf16 values in 340 tensors, with
    // their scaling: 826 us, 154 on one).
    ahead();
    const int end = static_cast<int>(left < chunk_values(VEC) ? left : chunk_values(VEC));
    for (int at = threadIdx.x; at < end; at += kClipThreads) {
      const float v = SCALED ? static_cast<float>(in[at]) * f : static_cast<float>(in[at]);
      a = ffma2(f32x2(v, 0.f), f32x2(v, 0.f), a);
    }
  }
  a = fadd2(a, b);
  return f32x2_lo(a) + f32x2_hi(a);
}

template <int VEC, typename T, typename Ahead>
SPARGE_DEV void add_chunk(const T* in, int64_t left, const Ahead& ahead, Sum& sum) {
  const float s = chunk_squares<VEC, false>(in, left, 1.f, ahead);
  if (s > 8.0779357e-28f && s < 2.1267648e37f) {  // 2^-90, 2^124
    sum.add(s);
    return;
  }
  // Out of range, or zeros: once more with the values brought into range.  Below,
  // all of them are under 2^-45, and 2^100 keeps the smallest from vanishing;
  // above, 2^-70 keeps the largest from overflowing, and what vanishes does not
  // matter beside it.
  const bool small = s < 1.f;
  const float again =
      chunk_squares<VEC, true>(in, left, small ? 1.2676506e30f : 8.4703295e-22f, [] {});
  sum.total += static_cast<double>(again) * (small ? 0x1p-200 : 0x1p140);
}

SPARGE_DEV double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int MAX, int VEC>
__global__ void __launch_bounds__(kClipThreads, 3) clip_norm_kernel(
    const __grid_constant__ ClipList<MAX> l, double* sums) {
  __shared__ double red[kClipThreads / 32];
  grid_launch_dependents();
  const uint32_t total = l.chunk[l.n];
  Sum sum;
  Chunk c = {};
  if (blockIdx.x < total) c = find<VEC>(l, blockIdx.x, 0, l.n);
  for (uint32_t k = blockIdx.x; k < total; k += gridDim.x) {
    const Chunk now = c;
    const auto ahead = [&] {
      if (k + gridDim.x < total) c = find<VEC>(l, k + gridDim.x, now.i, l.n);
    };
    if (l.bf16[now.i])
      add_chunk<VEC>(static_cast<const __nv_bfloat16*>(l.in[now.i]) + now.base, now.left, ahead, sum);
    else
      add_chunk<VEC>(static_cast<const float*>(l.in[now.i]) + now.base, now.left, ahead, sum);
  }
  sum.flush();
  double acc = warp_sum(sum.total);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kClipThreads / 32; ++w) acc += red[w];
    sums[blockIdx.x] = acc;
  }
}

template <int VEC, typename T, typename Ahead>
SPARGE_DEV void scale_chunk(const T* in, T* out, int64_t left, float c, const Ahead& ahead) {
  if (((reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) & 15) == 0) {
    Raw8<T> r[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const int at = place(k);
      const uint4* p = reinterpret_cast<const uint4*>(in + at);
#pragma unroll
      for (int i = 0; i < pieces8<T>(); ++i)
        r[k].v[i] = at + 8 <= left ? p[i] : make_uint4(0, 0, 0, 0);
    }
    ahead();
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      float f[8];
      unpack8(r[k], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= c;
      if (place(k) + 8 <= left) store8(out + place(k), f);
    }
    const int64_t whole = left & ~int64_t(7);
    if (left < chunk_values(VEC) && threadIdx.x < left - whole)
      out[whole + threadIdx.x] = static_cast<T>(static_cast<float>(in[whole + threadIdx.x]) * c);
  } else {
    ahead();
    const int end = static_cast<int>(left < chunk_values(VEC) ? left : chunk_values(VEC));
    for (int at = threadIdx.x; at < end; at += kClipThreads)
      out[at] = static_cast<T>(static_cast<float>(in[at]) * c);
  }
}

template <int MAX, int VEC>
__global__ void __launch_bounds__(kClipThreads, 3) clip_scale_kernel(
    const __grid_constant__ ClipList<MAX> l, const ClipArgs a) {
  __shared__ float factor;
  const uint32_t total = l.chunk[l.n];
  const bool writes = a.max_norm >= 0.f;
  Chunk c = {};
  if (writes && blockIdx.x < total) c = find<VEC>(l, total - 1 - blockIdx.x, 0, l.n);
  grid_wait();
  if (threadIdx.x < 32) {
    double v = 0.0;
    for (int i = threadIdx.x; i < a.n_sums; i += 32) v += a.sums[i];
    v = warp_sum(v);
    if (threadIdx.x == 0) {
      const double norm = sqrt(v);
      if (a.norm != nullptr && blockIdx.x == 0) *a.norm = static_cast<float>(norm);
      const double over = norm + static_cast<double>(a.eps);
      const double ratio = over == 0.0 ? 1.0 : static_cast<double>(a.max_norm) / over;
      factor = ratio > 1.0 ? 1.f : static_cast<float>(ratio);  // NaN stays NaN
    }
  }
  if (!writes) return;  // the norm alone
  __syncthreads();
  const float f = factor;
  if (a.in_place && f == 1.f) return;
  for (uint32_t k = blockIdx.x; k < total; k += gridDim.x) {
    const Chunk now = c;
    const auto ahead = [&] {
      if (k + gridDim.x < total) c = find<VEC>(l, total - 1 - k - gridDim.x, 0, now.i + 1);
    };
    if (l.bf16[now.i])
      scale_chunk<VEC>(static_cast<const __nv_bfloat16*>(l.in[now.i]) + now.base,
                  static_cast<__nv_bfloat16*>(l.out[now.i]) + now.base, now.left, f, ahead);
    else
      scale_chunk<VEC>(static_cast<const float*>(l.in[now.i]) + now.base,
                  static_cast<float*>(l.out[now.i]) + now.base, now.left, f, ahead);
  }
}

constexpr int64_t kMaxValues = int64_t(1) << 40;  // of one tensor

// Fills a list with tensors [first, first + count).
template <int MAX>
void fill(ClipList<MAX>& l, const sparge_tensor* t, void* const* out, int count, int vectors) {
  uint32_t chunks = 0;
  const int64_t values = chunk_values(vectors);
  for (int i = 0; i < count; ++i) {
    l.in[i] = t[i].data;
    l.out[i] = out != nullptr ? out[i] : t[i].data;
    l.numel[i] = t[i].numel;
    l.bf16[i] = t[i].type == SPARGE_BF16;
    l.chunk[i] = chunks;
    chunks += static_cast<uint32_t>((t[i].numel + values - 1) / values);
  }
  l.chunk[count] = chunks;
  l.n = count;
}

int list_vectors(const sparge_tensor* t, int count) {
  int64_t total = 0;
  for (int i = 0; i < count; ++i) total += t[i].numel;
  return total < static_cast<int64_t>(kSMs) * chunk_values(kVectors) ? kFewVectors : kVectors;
}

int list_ctas(uint32_t chunks, int most) {
  return static_cast<int>(std::max<uint32_t>(1, std::min<uint32_t>(chunks, most)));
}

template <int MAX, int VEC>
cudaError_t launch_norm(const sparge_tensor* t, int count, double* sums, int* ctas,
                        cudaStream_t st) {
  ClipList<MAX> l;
  fill(l, t, nullptr, count, VEC);
  *ctas = list_ctas(l.chunk[count], kNormCtas);
  clip_norm_kernel<MAX, VEC><<<*ctas, kClipThreads, 0, st>>>(l, sums);
  return cudaGetLastError();
}

template <int MAX, int VEC>
cudaError_t launch_scale(const sparge_tensor* t, void* const* out, int count, const ClipArgs& a,
                         bool first, cudaStream_t st) {
  ClipList<MAX> l;
  fill(l, t, out, count, VEC);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.max_norm < 0.f ? 1 : list_ctas(l.chunk[count], kScaleCtas));
  cfg.blockDim = dim3(kClipThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = first ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, clip_scale_kernel<MAX, VEC>, l, a);
}

// Whether two tensors that are written share memory (or one is listed twice):
// their chunks would be scaled twice, or while another CTA reads them.
struct Range {
  uintptr_t begin, end;
  bool operator<(const Range& o) const { return begin < o.begin; }
};
int check_overlap(const sparge_tensor* t, void* const* out, int n) {
  Range* r = new (std::nothrow) Range[n > 0 ? n : 1];
  if (r == nullptr) return SPARGE_ERR_WORKSPACE;
  int m = 0;
  for (int i = 0; i < n; ++i) {
    if (t[i].numel == 0) continue;
    const uintptr_t b = reinterpret_cast<uintptr_t>(out != nullptr ? out[i] : t[i].data);
    r[m++] = {b, b + static_cast<uintptr_t>(t[i].numel) * (t[i].type == SPARGE_BF16 ? 2 : 4)};
  }
  std::sort(r, r + m);
  int rc = SPARGE_OK;
  for (int i = 1; i < m; ++i)
    if (r[i].begin < r[i - 1].end) rc = SPARGE_ERR_INVALID_ARG;
  if (rc == SPARGE_OK && out != nullptr) {
    // An output may be its own input, but lie on no other one.
    for (int i = 0; i < n && rc == SPARGE_OK; ++i) {
      if (t[i].numel == 0) continue;
      const uintptr_t b = reinterpret_cast<uintptr_t>(t[i].data);
      const uintptr_t e = b + static_cast<uintptr_t>(t[i].numel) * (t[i].type == SPARGE_BF16 ? 2 : 4);
      const Range key = {e, e};
      const Range* after = std::lower_bound(r, r + m, key);  // first that begins at e or later
      while (after != r) {
        --after;
        if (after->end <= b) break;
        if (after->begin != reinterpret_cast<uintptr_t>(out[i]) || after->begin != b) {
          rc = SPARGE_ERR_INVALID_ARG;
          break;
        }
      }
    }
  }
  delete[] r;
  return rc;
}

int check_clip(const sparge_tensor* t, void* const* out, int32_t n, float max_norm, float eps,
               const float* norm) {
  if (n < 0 || (n > 0 && t == nullptr)) return SPARGE_ERR_INVALID_ARG;
  if (n > SPARGE_MAX_TENSORS) return SPARGE_ERR_UNSUPPORTED;
  if (isnan(max_norm) || isinf(max_norm)) return SPARGE_ERR_INVALID_ARG;
  if (!isfinite(eps) || eps < 0.f) return SPARGE_ERR_INVALID_ARG;
  if (norm == nullptr) return SPARGE_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(norm) % 4 != 0) return SPARGE_ERR_MISALIGNED;
  int64_t total = 0;
  for (int i = 0; i < n; ++i) {
    if (t[i].type != SPARGE_BF16 && t[i].type != SPARGE_F32) return SPARGE_ERR_UNSUPPORTED;
    if (t[i].numel < 0) return SPARGE_ERR_INVALID_ARG;
    if (t[i].numel == 0) continue;
    if (t[i].numel > kMaxValues || (total += t[i].numel) > kMaxValues)
      return SPARGE_ERR_UNSUPPORTED;
    const uintptr_t size = t[i].type == SPARGE_BF16 ? 2 : 4;
    if (t[i].data == nullptr || (out != nullptr && out[i] == nullptr))
      return SPARGE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(t[i].data) % size != 0 ||
        (out != nullptr && reinterpret_cast<uintptr_t>(out[i]) % size != 0))
      return SPARGE_ERR_MISALIGNED;
  }
  return max_norm < 0.f ? SPARGE_OK : check_overlap(t, out, n);
}

int lists_of(int n) { return n <= 0 ? 1 : (n + kLargeList - 1) / kLargeList; }

}  // namespace

}  // namespace sparge

using namespace sparge;

extern "C" {

int sparge_clip_workspace_bytes(int32_t n, size_t* bytes) {
  if (bytes == nullptr || n < 0) return SPARGE_ERR_INVALID_ARG;
  if (n > SPARGE_MAX_TENSORS) return SPARGE_ERR_UNSUPPORTED;
  *bytes = static_cast<size_t>(lists_of(n)) * kNormCtas * sizeof(double);
  return SPARGE_OK;
}

int sparge_clip_grads(const sparge_tensor* grads, void* const* out, int32_t n, float max_norm,
                      float eps, float* norm, void* workspace, size_t ws_bytes,
                      sparge_stream_t stream) {
  const int rc = check_clip(grads, out, n, max_norm, eps, norm);
  if (rc != SPARGE_OK) return rc;
  const int lists = lists_of(n);
  if (workspace == nullptr || ws_bytes < static_cast<size_t>(lists) * kNormCtas * sizeof(double))
    return SPARGE_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) % 16 != 0) return SPARGE_ERR_MISALIGNED;
  ClipArgs a = {};
  a.sums = static_cast<double*>(workspace);
  a.max_norm = max_norm;
  a.eps = eps;
  a.in_place = out == nullptr;
  for (int k = 0; k < lists; ++k) {
    const int first = k * kLargeList, count = std::min(n - first, kLargeList);
    int ctas = 0;
    const bool few = list_vectors(grads + first, count) == kFewVectors;
    const bool small = count <= kSmallList;
    auto* launch = few ? launch_norm<kSmallList, kFewVectors> : launch_norm<kSmallList, kVectors>;
    if (!small) launch = few ? launch_norm<kLargeList, kFewVectors> : launch_norm<kLargeList, kVectors>;
    const cudaError_t e = launch(grads + first, count, a.sums + a.n_sums, &ctas, stream);
    if (e != cudaSuccess) return SPARGE_ERR_CUDA;
    a.n_sums += ctas;
  }
  for (int k = 0; k < lists; ++k) {
    const int first = k * kLargeList, count = std::min(n - first, kLargeList);
    a.norm = k == 0 ? norm : nullptr;
    void* const* o = out != nullptr ? out + first : nullptr;
    const bool few = list_vectors(grads + first, count) == kFewVectors;
    auto* launch =
        count <= kSmallList
            ? (few ? launch_scale<kSmallList, kFewVectors> : launch_scale<kSmallList, kVectors>)
            : (few ? launch_scale<kLargeList, kFewVectors> : launch_scale<kLargeList, kVectors>);
    const cudaError_t e = launch(grads + first, o, count, a, k == 0, stream);
    if (e != cudaSuccess) return SPARGE_ERR_CUDA;
    if (max_norm < 0.f) break;
  }
  return SPARGE_OK;
}

}  // extern "C"
