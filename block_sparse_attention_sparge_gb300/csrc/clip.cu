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
// A thread squares and adds 32 values in fp32, then adds that to an fp64 sum.
// Where the fp32 sum left the range in which no square that matters over- or
// underflows (below 2^-90 or above 2^126), those 32 values are done again in
// fp64, so gradients of any size that fp32 holds give a finite norm of full
// precision.  An fp64 operation for every value instead would cap the pass
// below the memory's rate (fp64 runs at 1/60 of the fp32 rate here).
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

constexpr int kClipThreads = 512;
constexpr int kChunk = kClipThreads * 32;  // values a CTA takes at a time
constexpr int kClipCtas = kSMs * 4;        // sums of one launch in the workspace
constexpr int kSmallList = 48, kLargeList = 1024;  // tensors of one launch

// A list of tensors as a kernel parameter (27.7 KB of the 32 KB there is for
// the large one; the small one keeps short lists cheap to launch).
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

// The tensor that owns chunk c, by bisection of the chunk starts.
template <int MAX>
SPARGE_DEV int owner(const ClipList<MAX>& l, uint32_t c) {
  int lo = 0, hi = l.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (l.chunk[mid] <= c) lo = mid;
    else hi = mid;
  }
  return lo;
}

SPARGE_DEV double sum_squares(const float (&v)[32]) {
  uint64_t a = 0, b = 0;
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const uint64_t p = f32x2(v[i], v[i + 1]), q = f32x2(v[i + 2], v[i + 3]);
    a = ffma2(p, p, a);
    b = ffma2(q, q, b);
  }
  a = fadd2(a, b);
  const float s = f32x2_lo(a) + f32x2_hi(a);
  if (s > 8.0779357e-28f && s < 8.5070592e37f) return s;  // 2^-90, 2^126
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) any |= __float_as_uint(v[i]) & 0x7fffffffu;
  if (any == 0) return 0.0;
  double d = 0.0;
#pragma unroll 1
  for (int i = 0; i < 32; ++i) {
    // a dynamic index would send v to local memory
    float x = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) x = k == i ? v[k] : x;
    d += static_cast<double>(x) * static_cast<double>(x);
  }
  return d;
}

// 32 values of this thread from the chunk that starts at `base`: four groups
// of eight consecutive ones, zeros behind the end.
template <typename T>
SPARGE_DEV void load_chunk(const T* in, int64_t left, bool wide, float (&v)[32]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int at = (k * kClipThreads + threadIdx.x) * 8;
    float f[8];
    if (wide && at + 8 <= left) {
      unpack8(load8(in + at), f);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = at + i < left ? static_cast<float>(in[at + i]) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[8 * k + i] = f[i];
  }
}

// Sum over the CTA's threads, the same bits in every thread.
SPARGE_DEV double cta_sum(double v, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kClipThreads / 32; ++w) s += red[w];
  return s;
}

template <int MAX>
__global__ void __launch_bounds__(kClipThreads, 2) clip_norm_kernel(
    const __grid_constant__ ClipList<MAX> l, double* sums) {
  __shared__ double red[kClipThreads / 32];
  grid_launch_dependents();
  double acc = 0.0;
  for (uint32_t c = blockIdx.x; c < l.chunk[l.n]; c += gridDim.x) {
    const int i = owner(l, c);
    const int64_t base = static_cast<int64_t>(c - l.chunk[i]) * kChunk;
    const int64_t left = l.numel[i] - base;
    const bool wide = (reinterpret_cast<uintptr_t>(l.in[i]) & 15) == 0;
    float v[32];
    if (l.bf16[i])
      load_chunk(static_cast<const __nv_bfloat16*>(l.in[i]) + base, left, wide, v);
    else
      load_chunk(static_cast<const float*>(l.in[i]) + base, left, wide, v);
    acc += sum_squares(v);
  }
  acc = cta_sum(acc, red);
  if (threadIdx.x == 0) sums[blockIdx.x] = acc;
}

template <typename T>
SPARGE_DEV void scale_chunk(const T* in, T* out, int64_t left, float c) {
  const bool wide =
      ((reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) & 15) == 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int at = (k * kClipThreads + threadIdx.x) * 8;
    if (wide && at + 8 <= left) {
      Raw8<T> r;
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
        r.v[i] = reinterpret_cast<const uint4*>(in + at)[i];
      float f[8];
      unpack8(r, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= c;
      store8(out + at, f);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (at + i < left) out[at + i] = static_cast<T>(static_cast<float>(in[at + i]) * c);
    }
  }
}

template <int MAX>
__global__ void __launch_bounds__(kClipThreads, 2) clip_scale_kernel(
    const __grid_constant__ ClipList<MAX> l, const ClipArgs a) {
  __shared__ double red[kClipThreads / 32];
  grid_wait();
  double v = 0.0;
  for (int i = threadIdx.x; i < a.n_sums; i += kClipThreads) v += a.sums[i];
  const double norm = sqrt(cta_sum(v, red));
  if (a.norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = static_cast<float>(norm);
  if (a.max_norm < 0.f) return;  // the norm alone
  const double ratio = static_cast<double>(a.max_norm) / (norm + static_cast<double>(a.eps));
  const float c = ratio > 1.0 ? 1.f : static_cast<float>(ratio);  // NaN stays NaN
  if (a.in_place && c == 1.f) return;
  const uint32_t total = l.chunk[l.n];
  for (uint32_t k = blockIdx.x; k < total; k += gridDim.x) {
    const uint32_t ch = total - 1 - k;
    const int i = owner(l, ch);
    const int64_t base = static_cast<int64_t>(ch - l.chunk[i]) * kChunk;
    const int64_t left = l.numel[i] - base;
    if (l.bf16[i])
      scale_chunk(static_cast<const __nv_bfloat16*>(l.in[i]) + base,
                  static_cast<__nv_bfloat16*>(l.out[i]) + base, left, c);
    else
      scale_chunk(static_cast<const float*>(l.in[i]) + base, static_cast<float*>(l.out[i]) + base,
                  left, c);
  }
}

constexpr int64_t kMaxValues = int64_t(1) << 40;  // of one tensor

// Fills a list with tensors [first, first + count).
template <int MAX>
void fill(ClipList<MAX>& l, const sparge_tensor* t, void* const* out, int count) {
  uint32_t chunks = 0;
  for (int i = 0; i < count; ++i) {
    l.in[i] = t[i].data;
    l.out[i] = out != nullptr ? out[i] : t[i].data;
    l.numel[i] = t[i].numel;
    l.bf16[i] = t[i].type == SPARGE_BF16;
    l.chunk[i] = chunks;
    chunks += static_cast<uint32_t>((t[i].numel + kChunk - 1) / kChunk);
  }
  l.chunk[count] = chunks;
  l.n = count;
}

int list_ctas(uint32_t chunks) {
  return static_cast<int>(std::max<uint32_t>(1, std::min<uint32_t>(chunks, kClipCtas)));
}

template <int MAX>
cudaError_t launch_norm(const sparge_tensor* t, int count, double* sums, int* ctas,
                        cudaStream_t st) {
  ClipList<MAX> l;
  fill(l, t, nullptr, count);
  *ctas = list_ctas(l.chunk[count]);
  clip_norm_kernel<MAX><<<*ctas, kClipThreads, 0, st>>>(l, sums);
  return cudaGetLastError();
}

template <int MAX>
cudaError_t launch_scale(const sparge_tensor* t, void* const* out, int count, const ClipArgs& a,
                         bool first, cudaStream_t st) {
  ClipList<MAX> l;
  fill(l, t, out, count);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.max_norm < 0.f ? 1 : list_ctas(l.chunk[count]));
  cfg.blockDim = dim3(kClipThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = first ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, clip_scale_kernel<MAX>, l, a);
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
  *bytes = static_cast<size_t>(lists_of(n)) * kClipCtas * sizeof(double);
  return SPARGE_OK;
}

int sparge_clip_grads(const sparge_tensor* grads, void* const* out, int32_t n, float max_norm,
                      float eps, float* norm, void* workspace, size_t ws_bytes,
                      sparge_stream_t stream) {
  const int rc = check_clip(grads, out, n, max_norm, eps, norm);
  if (rc != SPARGE_OK) return rc;
  const int lists = lists_of(n);
  if (workspace == nullptr || ws_bytes < static_cast<size_t>(lists) * kClipCtas * sizeof(double))
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
    const cudaError_t e =
        count <= kSmallList
            ? launch_norm<kSmallList>(grads + first, count, a.sums + a.n_sums, &ctas, stream)
            : launch_norm<kLargeList>(grads + first, count, a.sums + a.n_sums, &ctas, stream);
    if (e != cudaSuccess) return SPARGE_ERR_CUDA;
    a.n_sums += ctas;
  }
  for (int k = 0; k < lists; ++k) {
    const int first = k * kLargeList, count = std::min(n - first, kLargeList);
    a.norm = k == 0 ? norm : nullptr;
    void* const* o = out != nullptr ? out + first : nullptr;
    const cudaError_t e =
        count <= kSmallList
            ? launch_scale<kSmallList>(grads + first, o, count, a, k == 0, stream)
            : launch_scale<kLargeList>(grads + first, o, count, a, k == 0, stream);
    if (e != cudaSuccess) return SPARGE_ERR_CUDA;
    if (max_norm < 0.f) break;
  }
  return SPARGE_OK;
}

}  // extern "C"
