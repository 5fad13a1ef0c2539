// Orthogonalised updates on sm_103a: the Newton-Schulz iteration
//   X = U / (|U| + eps),  X <- a X + B X,  B = b A + c A A,  A = X X^T
// over a list of matrices, X the short side by the long one (tall matrices are
// worked on transposed).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <vector>

#include "common.cuh"
#include "kernels.h"
#include "places.h"
#include "rows.cuh"
#include "sparge.h"

namespace sparge {

namespace {

// ------------------------------------------------------------------- layout
// X, A and B lie in the workspace as tiles of 128 rows x 64 columns of fp16, 16 KB
// each, rows of 128 bytes with the 16-byte pieces swizzled as the tensor cores read
// them: every operand tile is one contiguous copy, as it stands.  Rows and columns
// are padded with zeros to multiples of 128, which stay zeros through the products.
// A tile of fp32 values (X of the exact form) is 32 KB, its rows 256 bytes.
constexpr int kTR = 128, kTC = 64;
constexpr uint32_t kTile = kTR * kTC * 2;

// Scales (powers of two) that keep the fp16 values away from fp16's subnormals: the
// values of A and B, whose sizes are some units at most; those of X by the root of
// its columns, so that they are near one when the rows have norm one.
constexpr float kScaleA = 256.f;
inline int x_exponent(int n) { return static_cast<int>(lround(log2(static_cast<double>(n)) / 2)); }

constexpr int kMaxBatch = 64;
constexpr int64_t kMaxValues = int64_t(1) << 27;  // of a batch
constexpr int kNormParts = 256;                   // partial sums of a matrix

// A matrix as the products see it.  Offsets are in tiles of 16 KB from the base.
struct Shape {
  int mb, nb;        // blocks of 128 rows and columns of X
  int end_a, end_x;  // running count of output tiles: of A and B, of X
  int end_g;         // running count of the items of A = X X^T: tiles times parts
  int parts;         // of the contraction of A = X X^T
  uint32_t slot;     // its first partial sum, where there are several parts
  uint32_t count;    // and its first counter
  uint32_t x[2], a, b;
  uint32_t v;        // fp32 vectors: see below
  int kx;            // exponent of X's scale
};
struct ShapeBatch {
  int n;
  Shape s[kMaxBatch];
};

// A matrix as the first and last kernels see it.
struct Matrix {
  const void* grad;
  float* mom;
  void* out;
  int64_t gs, ms, os;
  int rows, cols;
  float keep, step;
  int grad_f32, out_f32, tall;
  int nb;             // blocks of 128 columns of X
  int end_p, end_t;   // running counts: CTAs of the norm, tiles of X
  uint32_t x0, xn;    // X at the start and at the end
  uint32_t v;
  int parts, part0;   // partial sums of the norm
  int kx;
};
struct MatrixBatch {
  int n;
  uint8_t* base;
  double* partial;
  int* counts;  // of the parts of A = X X^T that are done
  int n_counts;
  float mu, eps;
  int nesterov, update;
  Matrix m[kMaxBatch];
};

// Diagonals.  A and B are near multiples of the identity once X's rows have norm one,
// and what rounding takes from those (fp16's, and the tensor cores', which round
// sums towards zero at each addition) is what the result is off by.  So the
// diagonals are kept apart, in fp32, and the tiles of A and B hold zeros there:
// with A = D + E,
//   d_i = sum of row i's squares of X,
//   B_ij = E_ij (b + c (d_i + d_j)) + c (E E)_ij,   B_ii = b d_i + c (d_i^2 + (E E)_ii),
//   X_i <- (a + B_ii) X_i + sum over k != i of B_ik X_k.
// The squares come from whoever writes X, a sum for each row of each tile.
// Vectors of a matrix, from v on: [2 nb] of the sums of squares of X as stored
// (scaled by 4^kx), then d, then B_ii, each of 128 mb values.
SPARGE_DEV float* vectors(uint8_t* base, uint32_t v) {
  return reinterpret_cast<float*>(base + static_cast<int64_t>(v) * kTile);
}

// Tiles of a value's form: hi (fp16), then lo (fp16), then, in the exact form, fp32.
// Each plane of X holds mb * 2 nb tiles.
template <bool EXACT>
__host__ __device__ constexpr int x_planes() { return EXACT ? 4 : 2; }  // in tiles of 16 KB
template <bool EXACT>
__host__ __device__ constexpr int a_planes() { return EXACT ? 2 : 1; }

// Byte offset of the 16-byte piece ch (eight values) of row r in a tile.
SPARGE_DEV uint32_t piece(int r, int ch) { return r * 128 + ((ch ^ (r & 7)) << 4); }

// The same in a tile of fp32 values (four to a piece).
SPARGE_DEV uint32_t piece32(int r, int ch) { return r * 256 + ((ch ^ (r & 7)) << 4); }

SPARGE_DEV uint32_t pack_half2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
SPARGE_DEV void unpack_half8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = v.x, f[2 * i + 1] = v.y;
  }
}
// f to fp16 pairs: hi = fp16(f), lo = fp16(f - hi); hi + lo is off by 2^-22 of f at
// most (while lo is no subnormal).
SPARGE_DEV void split_half8(const float (&f)[8], uint4& hi, uint4& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = pack_half2(f[2 * i], f[2 * i + 1]);
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    l[i] = pack_half2(f[2 * i] - v.x, f[2 * i + 1] - v.y);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// Eight values of X (a piece of a tile) out of and into its planes, `plane` bytes apart.
template <bool EXACT>
SPARGE_DEV void load_x(const uint8_t* tiles, int64_t tile, int64_t plane, int r, int ch,
                       float (&f)[8]) {
  if constexpr (EXACT) {
    const uint8_t* p = tiles + 2 * plane + tile * 2 * kTile;
    const float4 u = __ldcg(reinterpret_cast<const float4*>(p + piece32(r, 2 * ch)));
    const float4 v = __ldcg(reinterpret_cast<const float4*>(p + piece32(r, 2 * ch + 1)));
    f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w;
    f[4] = v.x, f[5] = v.y, f[6] = v.z, f[7] = v.w;
  } else {
    const uint8_t* p = tiles + tile * kTile + piece(r, ch);
    float lo[8];
    unpack_half8(__ldcg(reinterpret_cast<const uint4*>(p)), f);
    unpack_half8(__ldcg(reinterpret_cast<const uint4*>(p + plane)), lo);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] += lo[i];
  }
}
template <bool EXACT>
SPARGE_DEV void store_x(uint8_t* tiles, int64_t tile, int64_t plane, int r, int ch,
                        const float (&f)[8]) {
  uint4 hi, lo;
  split_half8(f, hi, lo);
  uint8_t* p = tiles + tile * kTile + piece(r, ch);
  *reinterpret_cast<uint4*>(p) = hi;
  *reinterpret_cast<uint4*>(p + plane) = lo;
  if constexpr (EXACT) {
    uint8_t* q = tiles + 2 * plane + tile * 2 * kTile;
    *reinterpret_cast<float4*>(q + piece32(r, 2 * ch)) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(q + piece32(r, 2 * ch + 1)) = make_float4(f[4], f[5], f[6], f[7]);
  }
}

// --------------------------------------------------- the matrices themselves
// Eight values of a row from column c on (0 behind the last); 16-byte loads where
// the place allows them.  (Not through the read-only path: a momentum is written by the kernel
// before, which still runs when this one comes onto the machine, and a weight by this one.)
template <typename T>
SPARGE_DEV void read8(const T* row, int c, int cols, float (&f)[8]) {
  if (c + 8 <= cols && reinterpret_cast<uintptr_t>(row + c) % 16 == 0) {
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < pieces8<T>(); ++i) r.v[i] = reinterpret_cast<const uint4*>(row + c)[i];
    unpack8(r, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = c + i < cols ? static_cast<float>(row[c + i]) : 0.f;
  }
}
template <typename T>
SPARGE_DEV void write8(T* row, int c, int cols, const float (&f)[8]) {
  if (c + 8 <= cols && reinterpret_cast<uintptr_t>(row + c) % 16 == 0) {
    store8(row + c, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) row[c + i] = static_cast<T>(f[i]);
  }
}
SPARGE_DEV void read_any(const void* base, int f32, int64_t at, int c, int cols, float (&f)[8]) {
  if (f32)
    read8(static_cast<const float*>(base) + at, c, cols, f);
  else
    read8(static_cast<const __nv_bfloat16*>(base) + at, c, cols, f);
}
SPARGE_DEV void write_any(void* base, int f32, int64_t at, int c, int cols, const float (&f)[8]) {
  if (f32)
    write8(static_cast<float*>(base) + at, c, cols, f);
  else
    write8(static_cast<__nv_bfloat16*>(base) + at, c, cols, f);
}

// U at a row: the gradient, or with a momentum what the momentum (as stored) makes of it.
SPARGE_DEV void read_u(const MatrixBatch& p, const Matrix& m, int r, int c, float (&u)[8]) {
  read_any(m.grad, m.grad_f32, r * m.gs, c, m.cols, u);
  if (m.mom == nullptr) return;
  float v[8];
  read8(m.mom + r * m.ms, c, m.cols, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = p.nesterov ? fmaf(p.mu, v[i], u[i]) : v[i];
}

template <typename End>
SPARGE_DEV int find(int n, int at, End end) {  // the first i with at < end(i)
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (at < end(mid)) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// Squares of any size: those of values near one as they are, the others scaled.
// At most kSquares of them, then out into fp64, whose additions run at 1 / 64 of fp32's
// rate.
constexpr int kSquares = 64;
struct Squares {
  float big = 0.f, mid = 0.f, small = 0.f;
  SPARGE_DEV void add(const float (&x)[8]) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
    if (top >= 0x1p-40f && top <= 0x1p40f) {  // what is far below the largest may vanish
#pragma unroll
      for (int i = 0; i < 8; ++i) mid = fmaf(x[i], x[i], mid);
    } else {
#pragma unroll 1
      for (int i = 0; i < 8; ++i) add_any(x[i]);
    }
  }
  SPARGE_DEV void add_any(float x) {
    const float a = fabsf(x);
    if (a > 0x1p40f) {
      big = fmaf(x * 0x1p-70f, x * 0x1p-70f, big);
    } else if (a < 0x1p-40f) {
      small = fmaf(x * 0x1p100f, x * 0x1p100f, small);
    } else {
      mid = fmaf(x, x, mid);  // NaN too
    }
  }
  SPARGE_DEV void out(double& sum) {
    sum += mid;
    if (big != 0.f) sum += static_cast<double>(big) * 0x1p140;
    if (small != 0.f) sum += static_cast<double>(small) * 0x1p-200;
    big = mid = small = 0.f;
  }
};

// Sum over the 256 threads of a CTA, in a fixed order, for thread 0.
SPARGE_DEV double cta_sum(double v) {
  __shared__ double part[8];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();  // the last call's were read
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
    for (int i = 0; i < 8; ++i) s += part[i];
  return s;
}

// The momentum's step and the partial sums of U^2.  A CTA takes every parts-th
// piece of 16 rows x 128 columns, kAtOnce of them in flight.
constexpr int kAtOnce = 2;
__global__ void __launch_bounds__(256, 4) ortho_norm_kernel(const __grid_constant__ MatrixBatch p) {
  grid_launch_dependents();
  grid_wait();
  const int i = find(p.n, blockIdx.x, [&](int k) { return p.m[k].end_p; });
  const Matrix& m = p.m[i];
  const int part = blockIdx.x - (m.end_p - m.parts);
  const int across = (m.cols + 127) / 128;
  const int pieces = (m.rows + 15) / 16 * across;
  double sum = 0.0;
  Squares s;
  int n = 0;
  for (int q0 = part; q0 < pieces; q0 += kAtOnce * m.parts) {
    float u[kAtOnce][8], v[kAtOnce][8];
    int r[kAtOnce], c[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int q = q0 + k * m.parts;
      r[k] = q / across * 16 + threadIdx.x / 16;
      c[k] = q % across * 128 + threadIdx.x % 16 * 8;
      if (q >= pieces || r[k] >= m.rows) c[k] = m.cols;  // nothing there
      if (c[k] < m.cols) {
        read_any(m.grad, m.grad_f32, r[k] * m.gs, c[k], m.cols, u[k]);
        if (m.mom != nullptr) read8(m.mom + r[k] * m.ms, c[k], m.cols, v[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (c[k] >= m.cols) continue;
      if (m.mom != nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[k][j] = fmaf(p.mu, v[k][j], u[k][j]);
          u[k][j] = p.nesterov ? fmaf(p.mu, v[k][j], u[k][j]) : v[k][j];
        }
        write8(m.mom + r[k] * m.ms, c[k], m.cols, v[k]);
      }
      s.add(u[k]);
    }
    n += 8 * kAtOnce;
    if (n >= kSquares) s.out(sum), n = 0;
  }
  s.out(sum);
  sum = cta_sum(sum);
  if (threadIdx.x == 0) p.partial[m.part0 + part] = sum;
}

constexpr int kPitch = kTC + 1;  // floats of a row of a transposed tile in shared memory

// X of the start: U / (|U| + eps) in its tiles.  A CTA takes tiles side by side, of
// one matrix mostly, whose factor it works out once.
constexpr int kStartCtas = 8 * kSMs;
template <bool EXACT>
__global__ void __launch_bounds__(256) ortho_start_kernel(const __grid_constant__ MatrixBatch p) {
  __shared__ float t[kTR * kPitch];
  __shared__ float factor[2];
  grid_launch_dependents();
  grid_wait();
  for (int i = blockIdx.x * 256 + threadIdx.x; i < p.n_counts; i += gridDim.x * 256) p.counts[i] = 0;
  const int64_t all = p.m[p.n - 1].end_t;
  const int first = static_cast<int>(all * blockIdx.x / gridDim.x);
  const int last = static_cast<int>(all * (blockIdx.x + 1) / gridDim.x);
  int i = -1;
  float f1 = 0.f, f2 = 0.f;
  for (int at = first; at < last; ++at) {
    if (i < 0 || at >= p.m[i].end_t) {
      i = find(p.n, at, [&](int k) { return p.m[k].end_t; });
      const Matrix& m = p.m[i];
      double sum = 0.0;
      for (int k = threadIdx.x; k < m.parts; k += 256) sum += __ldcg(p.partial + m.part0 + k);
      sum = cta_sum(sum);
      if (threadIdx.x == 0) {
        // 2^kx / (|U| + eps) as two factors, neither of which leaves fp32's range.
        const double inv = scalbn(1.0, m.kx) / (sqrt(sum) + static_cast<double>(p.eps));
        int e = 0;
        const double frac = frexp(inv, &e);
        const bool fine = inv > 0.0 && inv < 1e300;
        factor[0] = fine ? scalbnf(1.f, e / 2) : 1.f;
        factor[1] = fine ? scalbnf(static_cast<float>(frac), e - e / 2) : static_cast<float>(inv);
      }
      __syncthreads();
      f1 = factor[0], f2 = factor[1];
    }
    const Matrix& m = p.m[i];
    const int tiles = m.end_t - (i > 0 ? p.m[i - 1].end_t : 0);
    const int tile = at - (m.end_t - tiles);
    const int64_t plane = static_cast<int64_t>(tiles) * kTile;
    const int r0 = tile / (2 * m.nb) * kTR, c0 = tile % (2 * m.nb) * kTC;
    uint8_t* x = p.base + static_cast<int64_t>(m.x0) * kTile;
    if (m.tall) {
      // Rows of the tile are columns of the matrix: 64 rows of it, 128 columns.
      __syncthreads();  // the last tile was read
#pragma unroll
      for (int k = threadIdx.x; k < kTC * 16; k += 256) {
        const int r = c0 + k / 16, c = r0 + k % 16 * 8;
        float u[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (r < m.rows && c < m.cols) read_u(p, m, r, c, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) t[(k % 16 * 8 + j) * kPitch + k / 16] = u[j];
      }
      __syncthreads();
    }
#pragma unroll
    for (int k = threadIdx.x; k < kTR * 8; k += 256) {
      const int r = k / 8, ch = k % 8;
      float u[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (m.tall) {
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = t[r * kPitch + ch * 8 + j];
      } else if (r0 + r < m.rows && c0 + ch * 8 < m.cols) {
        read_u(p, m, r0 + r, c0 + ch * 8, u);
      }
      float squares = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[j] = u[j] * f1 * f2;
        squares = fmaf(u[j], u[j], squares);
      }
      store_x<EXACT>(x, tile, plane, r, ch, u);
      squares = sum_of_8(squares);  // the eight threads of a row
      if (ch == 0)
        vectors(p.base, m.v)[static_cast<int64_t>(tile % (2 * m.nb)) *
                                 (tiles / (2 * m.nb) * kTR) + r0 + r] = squares;
    }
  }
}

// The result out of the last X's tiles: X itself, or the weight's step.
template <bool EXACT>
__global__ void __launch_bounds__(256) ortho_finish_kernel(const __grid_constant__ MatrixBatch p) {
  __shared__ float t[kTR * kPitch];
  grid_wait();
  const int i = find(p.n, blockIdx.x, [&](int k) { return p.m[k].end_t; });
  const Matrix& m = p.m[i];
  const int tiles = m.end_t - (i > 0 ? p.m[i - 1].end_t : 0);
  const int tile = blockIdx.x - (m.end_t - tiles);
  const int64_t plane = static_cast<int64_t>(tiles) * kTile;
  const int r0 = tile / (2 * m.nb) * kTR, c0 = tile % (2 * m.nb) * kTC;
  const uint8_t* x = p.base + static_cast<int64_t>(m.xn) * kTile;
  const float back = scalbnf(1.f, -m.kx);
  auto put = [&](int r, int c, float (&f)[8]) {
    if (p.update) {
      float w[8];
      read_any(m.out, m.out_f32, r * m.os, c, m.cols, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = fmaf(-m.step, f[j], m.keep * w[j]);
    }
    write_any(m.out, m.out_f32, r * m.os, c, m.cols, f);
  };
  for (int k = threadIdx.x; k < kTR * 8; k += 256) {
    const int r = k / 8, ch = k % 8;
    if (!m.tall && (r0 + r >= m.rows || c0 + ch * 8 >= m.cols)) continue;
    float f[8];
    load_x<EXACT>(x, tile, plane, r, ch, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= back;
    if (m.tall) {
#pragma unroll
      for (int j = 0; j < 8; ++j) t[r * kPitch + ch * 8 + j] = f[j];
    } else {
      put(r0 + r, c0 + ch * 8, f);
    }
  }
  if (!m.tall) return;
  __syncthreads();
  for (int k = threadIdx.x; k < kTC * 16; k += 256) {
    const int r = c0 + k / 16, c = r0 + k % 16 * 8;
    if (r >= m.rows || c >= m.cols) continue;
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = t[(k % 16 * 8 + j) * kPitch + k / 16];
    put(r, c, f);
  }
}

// ----------------------------------------------------------------- products
enum Product { kGram, kSquare, kApply };  // A = X X^T;  B = b A + c A A;  X = a X + B X

// An output tile is 128 rows x 128 columns of one CTA (CG 1), or 256 rows of a pair
// of CTAs (CG 2) x 256 columns (128 in the exact form), where each loads its rows of
// A and half of B's columns: half the bytes for as many products.  The contraction
// runs in steps of 64.  A and B are symmetric: tiles below the diagonal's blocks are
// not computed, the others are written twice, as they are and transposed.
// Eight epilogue warps read one accumulator while the products fill the other.
//
// The contraction of A = X X^T runs over the long side.  Where the tiles are few for
// the machine it is cut into parts (plan_parts): an epilogue warp writes its 32 x 64
// sums, and the one that finds by its counter that it is the last reads those of all
// parts, adds them in the parts' order (so the result does not depend on which came
// last) and goes on with the tile.  Six odd matrices, the longest 16 x 5120, fp32:
// A takes 21 us a step, 55 without parts; the whole call 244 us and 387.
template <int CG, bool EXACT>
struct GemmCfg {
  static constexpr int BN = CG == 2 && !EXACT ? 256 : 128;
  static constexpr int kWarps = 8;  // epilogue
  static constexpr int kThreads = (kWarps + 2) * 32;
  static constexpr int kPlanes = EXACT ? 2 : 1;  // operands: hi, or hi and lo
  static constexpr uint32_t kA = kTile;
  static constexpr uint32_t kB = BN / CG * 128;
  static constexpr uint32_t kStage = kPlanes * (kA + kB);
  // An epilogue warp's own: 32 rows of a tile, in two planes of fp16 or one of fp32.
  static constexpr uint32_t kHold = 8192;
  static constexpr int kUnits = CG * BN / 64 * 4;  // partial sums of a tile
  static constexpr int NST = static_cast<int>((226 * 1024 - kWarps * kHold) / kStage);
  static constexpr uint32_t off_hold = NST * kStage;
  static constexpr uint32_t off_bar = off_hold + kWarps * kHold;
  static constexpr int B_F = 0;             // NST: a stage's tiles landed (of both CTAs)
  static constexpr int B_E = NST;           // NST: its products done
  static constexpr int B_AF = 2 * NST;      // 2: an accumulator complete
  static constexpr int B_AE = B_AF + 2;     // 2, all epilogue warps (of both CTAs): it was read
  static constexpr int B_H = B_AE + 2;      // kWarps: what the warp holds landed
  static constexpr int B_DONE = B_H + kWarps;
  static constexpr int NBAR = B_DONE + 1;
  static constexpr uint32_t off_slot = off_bar + NBAR * 8;
  static constexpr uint32_t bytes = off_slot + 16;
  // The tensor cores round a sum towards zero at each addition, so a long one drifts.
  // The exact form therefore reads its accumulators out every kChunk steps and adds
  // those in registers; the products with a lo, 2^-11 of the others, have an
  // accumulator of their own for the whole tile.
  static constexpr int kChunk = EXACT ? 4 : INT_MAX;
  static constexpr uint32_t tmem_cols = (EXACT ? 4 : 2) * BN;
};

constexpr int kUnit = 32 * 65;  // values of a partial sum: those of a warp, and the diagonal's

struct GemmParams {
  uint8_t* base;
  float* sums;       // partial sums
  int* counts;       // and how many of a tile's parts are there
  int tiles;         // or items
  int from;          // which of a matrix's two X is read; the other is written
  float a, b, c;
  int32_t* status;
};

struct GemmTile {
  const Shape* s;
  int rb, cb;   // first block of 128 rows, of 128 columns
  int from;     // first step of the contraction
  int steps;    // and their number
  int index;    // of the tile in its matrix
  int part;
};
// Output tiles of a matrix: all of X's, those of A that reach the diagonal or above.
template <int CG, bool EXACT>
__host__ __device__ inline int row_tiles(int mb) { return (mb + CG - 1) / CG; }
template <int CG, bool EXACT>
__host__ __device__ inline int col_tiles(int nb) {
  constexpr int CU = GemmCfg<CG, EXACT>::BN / 128;
  return (nb + CU - 1) / CU;
}
template <int CG, bool EXACT>
__host__ __device__ inline int first_col(int i) {  // of row i of A's tiles
  return i * CG / (GemmCfg<CG, EXACT>::BN / 128);
}
template <int CG, bool EXACT, Product KIND>
SPARGE_DEV GemmTile gemm_tile(const ShapeBatch& sb, int t) {
  constexpr int CU = GemmCfg<CG, EXACT>::BN / 128;
  auto end = [&](int k) {
    return KIND == kApply ? sb.s[k].end_x : KIND == kGram ? sb.s[k].end_g : sb.s[k].end_a;
  };
  const int i = find(sb.n, t, end);
  const Shape& s = sb.s[i];
  t -= i == 0 ? 0 : end(i - 1);
  GemmTile g;
  g.s = &s;
  g.from = g.part = 0;
  g.steps = 2 * (KIND == kGram ? s.nb : s.mb);
  if (KIND == kGram) {
    g.part = t % s.parts;
    t /= s.parts;
    g.from = g.steps * g.part / s.parts;
    g.steps = g.steps * (g.part + 1) / s.parts - g.from;
  }
  g.index = t;
  const int across = col_tiles<CG, EXACT>(KIND == kApply ? s.nb : s.mb);
  int row = 0;
  if (KIND == kApply) {
    row = t / across;
    t -= row * across;
  } else {
    for (int n; t >= (n = across - first_col<CG, EXACT>(row)); ++row) t -= n;
    t += first_col<CG, EXACT>(row);
  }
  g.rb = row * CG;
  g.cb = t * CU;
  return g;
}

template <int CG, bool EXACT, Product KIND>
__global__ void __launch_bounds__(GemmCfg<CG, EXACT>::kThreads, 1)
    ortho_gemm_kernel(const __grid_constant__ CUtensorMap tm128,
                      const __grid_constant__ CUtensorMap tm64,
                      const __grid_constant__ ShapeBatch sb, const __grid_constant__ GemmParams p) {
  using C = GemmCfg<CG, EXACT>;
  constexpr int BN = C::BN;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t s0 = smem_u32(smem_raw);
  auto bar = [&](int i) -> uint32_t { return s0 + C::off_bar + 8u * i; };
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem_raw + C::off_slot);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CG == 2 ? static_cast<int>(cluster_rank()) : 0;
  const int first_tile = blockIdx.x / CG, stride = gridDim.x / CG;
  constexpr int kProducer = C::kWarps, kIssuer = C::kWarps + 1;
  grid_launch_dependents();

  if (threadIdx.x == 0) {
    // (The swizzled tiles need 1024-byte alignment.)
    if ((s0 & 1023u) != 0u) report_error(p.status, SPARGE_ERR_CUDA);
    for (int i = 0; i < C::NBAR; ++i)
      mbar_init(bar(i), i == C::B_AE || i == C::B_AE + 1 ? C::kWarps * CG : 1);
    fence_barrier_init();
  }
  if (warp == kIssuer) {
    if constexpr (CG == 2) {
      tmem_alloc_pair(smem_u32(slot), C::tmem_cols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(slot), C::tmem_cols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();  // the other CTA's barriers are ready
  tc_fence_after();
  const uint32_t tmem = *slot;
  grid_wait();  // the operands are the previous kernel's

  const uint32_t x_in = p.from, x_out = p.from ^ 1;
  if (warp == kProducer) {
    if (lane == 0) {
      bool ok = true;
      int g = 0;
      for (int t = first_tile; ok && t < p.tiles; t += stride) {
        const GemmTile w = gemm_tile<CG, EXACT, KIND>(sb, t);
        const Shape& s = *w.s;
        const int mb = s.mb, xt = 2 * s.nb, at = 2 * mb;  // tiles of a row of X; of A
        const int nb = KIND == kApply ? s.nb : mb;         // blocks of columns of the output
        // Rows of 128 bytes from the base: X, and A or B.
        const int64_t X = static_cast<int64_t>(s.x[x_in]) * kTR;
        const int64_t A = static_cast<int64_t>(KIND == kSquare ? s.a : s.b) * kTR;
        const int64_t x_plane = static_cast<int64_t>(mb) * xt * kTR;
        const int64_t a_plane = static_cast<int64_t>(mb) * at * kTR;
        const int rb = w.rb + rank;
        const int both = min(CG, mb - w.rb);                   // CTAs with rows
        const int wide = min(BN / 128, nb - w.cb);             // blocks with columns
        const uint32_t bytes = C::kPlanes * (both * kTile + wide * kTile);
        for (int k = w.from; k < w.from + w.steps; ++k, ++g) {
          const int st = g % C::NST;
          if (g >= C::NST && !mbar_wait(bar(C::B_E + st), ((g / C::NST) - 1) & 1, kWaitTimeoutNs)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(bar(C::B_F + st), bytes);
          const uint32_t full = CG == 2 ? cluster_addr(bar(C::B_F + st), 0) : bar(C::B_F + st);
          auto load = [&](uint32_t dst, int64_t row, int rows) {
            if constexpr (CG == 2)
              tma_load_2d_pair(dst, rows == kTR ? &tm128 : &tm64, full, 0, static_cast<int>(row));
            else
              bulk_load(dst, p.base + row * 128, rows * 128, full);
          };
          for (int pl = 0; pl < C::kPlanes; ++pl) {
            const uint32_t da = s0 + st * C::kStage + pl * C::kA;
            const uint32_t db = s0 + st * C::kStage + C::kPlanes * C::kA + pl * C::kB;
            const int64_t xp = X + pl * x_plane, ap = A + pl * a_plane;
            if (rb < mb)
              load(da, KIND == kGram ? xp + static_cast<int64_t>(rb * xt + k) * kTR
                                     : ap + static_cast<int64_t>(rb * at + k) * kTR, kTR);
            if constexpr (KIND == kApply) {
              // 64 rows of X: half of each column's tile.
              constexpr int kCols = BN / CG / 64;
              for (int j = 0; j < kCols; ++j) {
                const int col = 2 * w.cb + rank * kCols + j;
                if (col < xt)
                  load(db + j * (kTile / 2),
                       xp + static_cast<int64_t>((k >> 1) * xt + col) * kTR + (k & 1) * 64, 64);
              }
            } else {
              // Rows of the other side: a block, or half of one.
              const int64_t from = KIND == kGram ? xp : ap;
              const int across = KIND == kGram ? xt : at;
              if constexpr (CG == 2 && BN == 128) {
                load(db, from + static_cast<int64_t>(w.cb * across + k) * kTR + rank * 64, 64);
              } else if (w.cb + rank < nb) {
                load(db, from + static_cast<int64_t>((w.cb + rank) * across + k) * kTR, kTR);
              }
            }
          }
        }
      }
      if (!ok) report_error(p.status, SPARGE_ERR_TIMEOUT);
      // Let the last copies land before the CTA can exit.
      if (rank == 0)
        for (int i = max(0, g - C::NST); i < g; ++i)
          mbar_wait(bar(C::B_F + i % C::NST), (i / C::NST) & 1, kWaitTimeoutNs);
    }
    __syncwarp();
  } else if (warp == kIssuer) {
    // The whole warp runs the loop; one elected lane issues each MMA.  B's rows are
    // the contraction's in kApply (MN-major), its columns in the others (K-major).
    constexpr uint32_t id = idesc_fp16(kTR * CG, BN, false, KIND == kApply);
    auto commit = [&](int i) {
      if constexpr (CG == 2) warp_commit_pair(bar(i));
      else warp_commit(bar(i));
    };
    bool ok = true;
    int g = 0, q = 0, odd = 0;
    for (int t = first_tile; rank == 0 && ok && t < p.tiles; t += stride, odd ^= 1) {
      const GemmTile w = gemm_tile<CG, EXACT, KIND>(sb, t);
      const uint32_t cross = tmem + (2 + odd) * BN;
      for (int k0 = 0; ok && k0 < w.steps; k0 += min(C::kChunk, w.steps - k0), ++q) {
        const int buf = q & 1;
        if (q >= 2 && !warp_wait_cluster(bar(C::B_AE + buf), ((q >> 1) - 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + buf * BN;
        const int n = min(C::kChunk, w.steps - k0);
        for (int k = 0; k < n; ++k, ++g) {
          const int st = g % C::NST;
          if (!warp_wait(bar(C::B_F + st), (g / C::NST) & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = s0 + st * C::kStage, sbb = sa + C::kPlanes * C::kA;
          // hi hi; hi lo and lo hi (lo lo is below what fp32 keeps).
#pragma unroll
          for (int pr = 0; pr < (EXACT ? 3 : 1); ++pr) {
            const uint64_t da = sdesc_sw128(sa + (pr == 2 ? C::kA : 0), 16, 1024);
            const uint64_t db = sdesc_sw128(sbb + (pr == 1 ? C::kB : 0),
                                            KIND == kApply ? kTile / 2 : 16, 1024);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint64_t dak = sdesc_add(da, kk * 32);
              const uint64_t dbk = sdesc_add(db, KIND == kApply ? kk * 2048 : kk * 32);
              const uint32_t add = (k > 0 || pr > 1 || kk > 0 || (pr == 1 && k0 > 0)) ? 1u : 0u;
              if constexpr (CG == 2) warp_mma_f16_pair(pr > 0 ? cross : d, dak, dbk, id, add);
              else warp_mma_bf16(pr > 0 ? cross : d, dak, dbk, id, add);
            }
          }
          commit(C::B_E + st);
        }
        if (ok) commit(C::B_AF + buf);
      }
    }
    if (!ok && lane == 0) report_error(p.status, SPARGE_ERR_TIMEOUT);
    if (rank == 0) {
      commit(C::B_DONE);
      warp_wait(bar(C::B_DONE), 0);
    }
  } else {
    // Thread = row r of the CTA's block (TMEM lane); the two warps of a quarter take
    // every other 64-column tile.  A warp's 32 rows of a tile are 4 KB in a row: they
    // come into what the warp holds, are changed there row by row, and go out again,
    // by bulk copies.
    const int quarter = warp & 3, half = warp >> 2;
    const int r = quarter * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    uint8_t* hold = smem_raw + C::off_hold + warp * C::kHold;
    const uint32_t hold_at = s0 + C::off_hold + warp * C::kHold;
    const uint32_t full = bar(C::B_H + warp);
    const uint32_t read_out = CG == 2 ? cluster_addr(bar(C::B_AE), 0) : bar(C::B_AE);
    constexpr uint32_t kPlane = kTile / 4;  // bytes of a warp's rows
    bool ok = true;
    int q = 0, odd = 0, held = 0;
    for (int t = first_tile; ok && t < p.tiles; t += stride, odd ^= 1) {
      const GemmTile w = gemm_tile<CG, EXACT, KIND>(sb, t);
      const Shape& s = *w.s;
      const int mb = s.mb, xt = 2 * s.nb, at = 2 * mb, rb = w.rb + rank;
      const int across = KIND == kApply ? xt : at;
      const int64_t x_plane = static_cast<int64_t>(mb) * xt * kTile;
      const int64_t a_plane = static_cast<int64_t>(mb) * at * kTile;
      const uint8_t* A = p.base + static_cast<int64_t>(s.a) * kTile;
      uint8_t* G = p.base + static_cast<int64_t>(KIND == kGram ? s.a : s.b) * kTile;
      const uint8_t* X = p.base + static_cast<int64_t>(s.x[x_in]) * kTile;
      uint8_t* Y = p.base + static_cast<int64_t>(s.x[x_out]) * kTile;
      // A = X X^T comes scaled by 4^kx, A A by kScaleA^2, B X by kScaleA.
      const float f = KIND == kGram     ? scalbnf(kScaleA, -2 * s.kx)
                      : KIND == kSquare ? p.c / kScaleA
                                        : 1.f / kScaleA;
      float* vec = vectors(p.base, s.v);
      const int64_t rows = static_cast<int64_t>(mb) * kTR;
      float* dA = vec + static_cast<int64_t>(xt) * rows;
      float* dB = dA + rows;
      const int row = rb * kTR + r;

      // Whether the j-th 64-column tile is there and this warp's to write.
      auto wanted = [&](int j) {
        return rb < mb && 2 * w.cb + j < across && (KIND == kApply || w.cb + j / 2 >= rb);
      };
      auto tile_of = [&](int j) { return static_cast<int64_t>(rb) * across + 2 * w.cb + j; };
      // What the warp holds is free again; the j-th tile's values on their way in.
      auto fetch = [&](int j) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          bulk_wait_read();
          if constexpr (KIND == kApply) {
            mbar_arrive_expect_tx(full, 2 * kPlane);
            if constexpr (EXACT) {
              bulk_load(hold_at, X + 2 * x_plane + tile_of(j) * 2 * kTile + quarter * 2 * kPlane,
                        2 * kPlane, full);
            } else {
              const uint8_t* src = X + tile_of(j) * kTile + quarter * kPlane;
              bulk_load(hold_at, src, kPlane, full);
              bulk_load(hold_at + kPlane, src + x_plane, kPlane, full);
            }
          } else if constexpr (KIND == kSquare) {
            mbar_arrive_expect_tx(full, C::kPlanes * kPlane);
            const uint8_t* src = A + tile_of(j) * kTile + quarter * kPlane;
            bulk_load(hold_at, src, kPlane, full);
            if constexpr (EXACT) bulk_load(hold_at + kPlane, src + a_plane, kPlane, full);
          }
        }
        __syncwarp();
      };
      auto held_piece = [&](int plane, int ch) -> uint4& {
        return *reinterpret_cast<uint4*>(hold + plane * kPlane + piece(lane, ch));
      };
      // The held planes are written: out with them.
      auto put_out = [&](uint8_t* dst, uint32_t from, uint32_t bytes) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          bulk_store(dst, hold_at + from, bytes);
          bulk_commit();
        }
      };
      auto diagonal = [&](int j) {  // whether the warp's rows of the j-th tile meet it
        const int col0 = (2 * w.cb + j) * kTC;
        return row - lane >= col0 && row - lane < col0 + kTC;
      };
      // A's diagonal, of this part's columns of X.
      auto squares_of = [&](int j) {
        float sum = 0.f;
        if (KIND == kGram && diagonal(j)) {
#pragma unroll 8
          for (int i = w.from; i < w.from + w.steps; ++i) sum += __ldcg(vec + i * rows + row);
        }
        return sum;
      };
      // A part's sums of the j-th tile to those of the whole contraction; false where
      // other parts are still to come.
      auto join = [&](int j, float (&y)[64], float& squares) {
        if (KIND != kGram || s.parts == 1) return true;
        const int64_t unit = (rank * (BN / 64) + j) * 4 + quarter;
        float* mine = p.sums + (s.slot + static_cast<int64_t>(w.index) * s.parts * C::kUnits + unit) *
                                   kUnit;
        constexpr int64_t kNext = static_cast<int64_t>(C::kUnits) * kUnit;
        float4* dst = reinterpret_cast<float4*>(mine + w.part * kNext);
#pragma unroll
        for (int e = 0; e < 16; ++e)
          __stcg(dst + e * 32 + lane, make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]));
        __stcg(mine + w.part * kNext + 64 * 32 + lane, squares);
        __threadfence();
        __syncwarp();
        int* count = p.counts + s.count + static_cast<int64_t>(w.index) * C::kUnits + unit;
        int before = lane == 0 ? atomicAdd(count, 1) : 0;
        before = __shfl_sync(0xffffffffu, before, 0);
        if (before != s.parts - 1) return false;
        __threadfence();
        if (lane == 0) *count = 0;  // for the next step
        squares = 0.f;
#pragma unroll
        for (int i = 0; i < 64; ++i) y[i] = 0.f;
        for (int q = 0; q < s.parts; ++q) {
          const float4* src = reinterpret_cast<const float4*>(mine + q * kNext);
          squares += __ldcg(mine + q * kNext + 64 * 32 + lane);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float4 u = __ldcg(src + e * 32 + lane);
            y[4 * e] += u.x, y[4 * e + 1] += u.y, y[4 * e + 2] += u.z, y[4 * e + 3] += u.w;
          }
        }
        return true;
      };
      // The products' sums of the j-th tile to its results.
      auto process = [&](int j, float (&y)[64], float diag) {
        const int64_t tile = tile_of(j);
        const int64_t at_byte = tile * kTile + quarter * kPlane;
        const int col0 = (2 * w.cb + j) * kTC;
#pragma unroll
        for (int i = 0; i < 64; ++i) y[i] *= f;
        if constexpr (KIND != kGram) {
          if (!warp_wait(full, held & 1)) ok = false;
          ++held;
        }
        if constexpr (KIND == kApply) {
          const float a_row = p.a + __ldcg(dB + row);
          float squares = 0.f;
#pragma unroll
          for (int ch = 0; ch < 8; ++ch) {
            float x[8], v[8];
            if constexpr (EXACT) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float4 u = *reinterpret_cast<float4*>(hold + piece32(lane, 2 * ch + e));
                x[4 * e] = u.x, x[4 * e + 1] = u.y, x[4 * e + 2] = u.z, x[4 * e + 3] = u.w;
              }
            } else {
              float lo[8];
              unpack_half8(held_piece(0, ch), x);
              unpack_half8(held_piece(1, ch), lo);
#pragma unroll
              for (int i = 0; i < 8; ++i) x[i] += lo[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              v[i] = y[8 * ch + i] = fmaf(a_row, x[i], y[8 * ch + i]);
              squares = fmaf(v[i], v[i], squares);
            }
            if constexpr (EXACT) {
#pragma unroll
              for (int e = 0; e < 2; ++e)
                *reinterpret_cast<float4*>(hold + piece32(lane, 2 * ch + e)) =
                    make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
            } else {
              split_half8(v, held_piece(0, ch), held_piece(1, ch));
            }
          }
          vec[(2 * w.cb + j) * rows + row] = squares;
          if constexpr (EXACT) {
            put_out(Y + 2 * x_plane + tile * 2 * kTile + quarter * 2 * kPlane, 0, 2 * kPlane);
            if (lane == 0) bulk_wait_read();
            __syncwarp();
#pragma unroll
            for (int ch = 0; ch < 8; ++ch) {
              float v[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] = y[8 * ch + i];
              split_half8(v, held_piece(0, ch), held_piece(1, ch));
            }
          }
          put_out(Y + at_byte, 0, kPlane);
          put_out(Y + x_plane + at_byte, kPlane, kPlane);
        } else {
          if constexpr (KIND == kSquare) {
            const float d_row = dA[row];
#pragma unroll
            for (int ch = 0; ch < 8; ++ch) {
              float e[8];
              unpack_half8(held_piece(0, ch), e);
              if constexpr (EXACT) {
                float lo[8];
                unpack_half8(held_piece(1, ch), lo);
#pragma unroll
                for (int i = 0; i < 8; ++i) e[i] += lo[i];
              }
              const float4 d0 = *reinterpret_cast<const float4*>(dA + col0 + 8 * ch);
              const float4 d1 = *reinterpret_cast<const float4*>(dA + col0 + 8 * ch + 4);
              const float d[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
#pragma unroll
              for (int i = 0; i < 8; ++i)
                y[8 * ch + i] = fmaf(e[i], fmaf(p.c, d_row + d[i], p.b), y[8 * ch + i]);
            }
          }
          if (diagonal(j)) {
            if constexpr (KIND == kGram) dA[row] = scalbnf(diag, -2 * s.kx);
#pragma unroll
            for (int i = 0; i < 64; ++i) {
              if (col0 + i != row) continue;
              if constexpr (KIND == kSquare) {
                const float d_row = dA[row];
                dB[row] = fmaf(d_row, fmaf(p.c, d_row, p.b), y[i] / kScaleA);
              }
              y[i] = 0.f;
            }
          }
          const int cbk = w.cb + j / 2;  // the tile's block of columns
#pragma unroll
          for (int pl = 0; pl < C::kPlanes; ++pl) {
            if (pl > 0 && lane == 0) bulk_wait_read();
            __syncwarp();  // every lane has read what it held
            uint32_t bits[32];
#pragma unroll
            for (int ch = 0; ch < 8; ++ch) {
              float v[8];
              uint4 hi, lo;
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] = y[8 * ch + i];
              split_half8(v, hi, lo);
              const uint4 u = pl == 0 ? hi : lo;
              held_piece(0, ch) = u;
              bits[4 * ch] = u.x, bits[4 * ch + 1] = u.y, bits[4 * ch + 2] = u.z, bits[4 * ch + 3] = u.w;
            }
            put_out(G + pl * a_plane + at_byte, 0, kPlane);
            if (cbk > rb) {
              // The same transposed, 32 columns at a time: each becomes 64 bytes of a row.
              constexpr int kPitch16 = 80;
              uint8_t* turn = hold + kPlane;
#pragma unroll
              for (int c0 = 0; c0 < 64; c0 += 32) {
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                  const uint32_t u = bits[(c0 + c) / 2];
                  *reinterpret_cast<uint16_t*>(turn + c * kPitch16 + lane * 2) = u & 0xffffu;
                  *reinterpret_cast<uint16_t*>(turn + (c + 1) * kPitch16 + lane * 2) = u >> 16;
                }
                __syncwarp();
                uint8_t* dst = G + pl * a_plane +
                               (static_cast<int64_t>(cbk) * at + 2 * rb + quarter / 2) * kTile;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  *reinterpret_cast<uint4*>(
                      dst + piece((j & 1) * 64 + c0 + lane, (quarter & 1) * 4 + e)) =
                      *reinterpret_cast<const uint4*>(turn + lane * kPitch16 + e * 16);
                __syncwarp();
              }
            }
          }
        }
      };
      // An accumulator was read.
      auto release = [&](int buf) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 2) mbar_arrive_cluster(read_out + 8u * buf);
          else mbar_arrive(bar(C::B_AE + buf));
        }
      };

      float acc[64];
      if constexpr (EXACT) {
        if (wanted(half)) fetch(half);
        for (int k0 = 0; k0 < w.steps; k0 += C::kChunk, ++q) {
          const int buf = q & 1;
          if (!warp_wait(bar(C::B_AF + buf), (q >> 1) & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const bool last = k0 + C::kChunk >= w.steps;
#pragma unroll
          for (int c0 = 0; c0 < 64; c0 += 32) {
            float v[32];
            tmem_ld32(lanes + buf * BN + half * 64 + c0, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[c0 + i] = k0 == 0 ? v[i] : acc[c0 + i] + v[i];
            if (last) {
              tmem_ld32(lanes + (2 + odd) * BN + half * 64 + c0, v);
#pragma unroll
              for (int i = 0; i < 32; ++i) acc[c0 + i] += v[i];
            }
          }
          release(buf);
        }
        if (ok && wanted(half)) {
          float diag = squares_of(half);
          if (join(half, acc, diag)) process(half, acc, diag);
        }
      } else {
        const int buf = q & 1;
        if (wanted(half)) fetch(half);
        if (!warp_wait(bar(C::B_AF + buf), (q >> 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll 1
        for (int j = half; j < BN / 64; j += 2) {
          if (wanted(j)) {
            if (j != half) fetch(j);
#pragma unroll
            for (int c0 = 0; c0 < 64; c0 += 32) {
              float v[32];
              tmem_ld32(lanes + buf * BN + j * 64 + c0, v);
#pragma unroll
              for (int i = 0; i < 32; ++i) acc[c0 + i] = v[i];
            }
          }
          if (j + 2 >= BN / 64) release(buf);
          if (wanted(j)) {
            float diag = squares_of(j);
            if (join(j, acc, diag)) process(j, acc, diag);
          }
        }
        ++q;
      }
    }
    if (!ok) report_error(p.status, SPARGE_ERR_TIMEOUT);
    if (lane == 0) bulk_wait();  // every result is out
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();  // neither CTA's memory is in use any more
  if (warp == kIssuer) {
    tc_fence_after();
    if constexpr (CG == 2) tmem_dealloc_pair(tmem, C::tmem_cols);
    else tmem_dealloc(tmem, C::tmem_cols);
  }
}

// -------------------------------------------------------------------- host
// A launch that may start while the kernel before it on the stream ends
// (programmatic dependent launch); every kernel here waits before it reads.
template <typename... Params>
cudaError_t launch_chained(void (*kernel)(Params...), int grid, int threads, uint32_t smem, int cluster,
                           cudaStream_t st, const Params&... params) {
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, params...);
}

int blocks_of(int n) { return (n + 127) / 128; }

// The matrices [at, end) of a list as one batch, and its workspace.
struct Batch {
  int end;
  ShapeBatch shapes;
  MatrixBatch mats;
  size_t bytes;        // tiles, then the partial sums of the norms, counters, those of A
  size_t sums;         // where the last begin
  int norm_ctas, tiles;
  int pairs;           // whether pairs of CTAs compute the products
  int tiles_a, tiles_x, items_g;
};

// Running counts of the output tiles; their totals for A and for X.
template <int CG, bool EXACT>
void count_tiles(ShapeBatch& sb, int& tiles_a, int& tiles_x) {
  tiles_a = tiles_x = 0;
  for (int k = 0; k < sb.n; ++k) {
    Shape& s = sb.s[k];
    const int down = row_tiles<CG, EXACT>(s.mb);
    for (int i = 0; i < down; ++i)
      tiles_a += col_tiles<CG, EXACT>(s.mb) - first_col<CG, EXACT>(i);
    tiles_x += down * col_tiles<CG, EXACT>(s.nb);
    s.end_a = tiles_a;
    s.end_x = tiles_x;
  }
}

// Pairs of CTAs where their tiles fill half of the machine, single CTAs else.
constexpr int kPairTiles = kSMs / 4;

// Cuts the contractions of A = X X^T: into parts of a number of steps for which the
// busiest CTA (items go round) is done first.  In steps of the products: an item
// costs kItemSteps beside its own, a join kJoinSteps for each part (reading 8 KB of
// sums a warp takes 0.7 us; a step 0.7 us in the exact form, 0.25 us in the other).
constexpr int kItemSteps = 4, kMaxParts = 64;
template <int CG, bool EXACT>
void plan_parts(Batch& b) {
  count_tiles<CG, EXACT>(b.shapes, b.tiles_a, b.tiles_x);
  constexpr int kJoinSteps = EXACT ? 1 : 3, kSlots = kSMs / CG;
  auto tiles_of = [&](int k) { return b.shapes.s[k].end_a - (k > 0 ? b.shapes.s[k - 1].end_a : 0); };
  auto parts_of = [&](int k, int steps) {
    return std::max(1, std::min(kMaxParts, (2 * b.shapes.s[k].nb + steps - 1) / steps));
  };
  int longest = 0;
  for (int k = 0; k < b.shapes.n; ++k) longest = std::max(longest, 2 * b.shapes.s[k].nb);
  int chosen = longest;
  if (b.tiles_a <= 2 * kSlots) {
    int64_t least = INT64_MAX;
    for (int steps = longest; steps >= 4; steps = steps * 3 / 4) {
      int load[kSlots] = {};
      int at = 0, items = 0;
      for (int k = 0; k < b.shapes.n; ++k) {
        const int parts = parts_of(k, steps);
        const int each = (2 * b.shapes.s[k].nb + parts - 1) / parts + kItemSteps +
                         (parts > 1 ? parts * kJoinSteps : 0);
        items += tiles_of(k) * parts;
        if (items > 2 * kSlots + b.tiles_a) break;
        for (int i = tiles_of(k) * parts; i > 0; --i, at = at + 1 < kSlots ? at + 1 : 0) load[at] += each;
      }
      if (items > 2 * kSlots + b.tiles_a) break;
      const int64_t most = *std::max_element(load, load + kSlots);
      if (most < least) least = most, chosen = steps;
    }
  }
  uint32_t slots = 0, counts = 0;
  for (int k = 0; k < b.shapes.n; ++k) {
    Shape& s = b.shapes.s[k];
    s.parts = parts_of(k, chosen);
    s.slot = slots;
    s.count = counts;
    b.items_g += tiles_of(k) * s.parts;
    s.end_g = b.items_g;
    if (s.parts == 1) continue;
    counts += tiles_of(k) * GemmCfg<CG, EXACT>::kUnits;
    slots += tiles_of(k) * s.parts * GemmCfg<CG, EXACT>::kUnits;
  }
  b.mats.n_counts = static_cast<int>(counts);
  b.sums = (b.bytes + counts * sizeof(int) + 255) / 256 * 256;
  b.mats.counts = reinterpret_cast<int*>(b.bytes);  // an offset, too
  b.bytes = b.sums + static_cast<size_t>(slots) * kUnit * sizeof(float);
}

Batch make_batch(const sparge_ortho& a, int at) {
  Batch b = {};
  const bool exact = !a.half;
  int64_t values = 0;
  uint32_t used = 0;  // tiles of 16 KB
  int partials = 0, i = at;
  for (; i < a.n && i - at < kMaxBatch; ++i) {
    const sparge_matrix& s = a.mats[i];
    const int rb = blocks_of(s.rows), cb = blocks_of(s.cols);
    const int64_t size = static_cast<int64_t>(rb) * cb * 128 * 128;
    if (i > at && values + size > kMaxValues) break;
    values += size;
    const int k = i - at;
    Shape& h = b.shapes.s[k];
    Matrix& m = b.mats.m[k];
    m.tall = s.rows > s.cols;
    h.mb = std::min(rb, cb);
    h.nb = std::max(rb, cb);
    h.kx = x_exponent(std::max(s.rows, s.cols));
    const uint32_t xt = static_cast<uint32_t>(h.mb) * 2 * h.nb, at_ = static_cast<uint32_t>(h.mb) * 2 * h.mb;
    for (int j = 0; j < 2; ++j) {
      h.x[j] = used;
      used += xt * (exact ? x_planes<true>() : x_planes<false>());
    }
    h.a = used;
    used += at_ * (exact ? a_planes<true>() : a_planes<false>());
    h.b = used;
    used += at_ * (exact ? a_planes<true>() : a_planes<false>());
    h.v = used;
    used += (static_cast<uint32_t>(h.mb) * (2 * h.nb + 2) * kTR * sizeof(float) + kTile - 1) / kTile;
    m.v = h.v;
    m.grad = s.grad;
    m.mom = s.momentum;
    m.out = s.out;
    m.gs = s.grad_stride;
    m.ms = s.momentum_stride;
    m.os = s.out_stride;
    m.rows = s.rows;
    m.cols = s.cols;
    m.keep = s.keep;
    m.step = s.step;
    m.grad_f32 = s.grad_type == SPARGE_F32;
    m.out_f32 = s.out_type == SPARGE_F32;
    m.nb = h.nb;
    m.kx = h.kx;
    m.parts = std::min(kNormParts, (s.rows + 15) / 16 * cb);
    m.part0 = partials;
    partials += m.parts;
    b.norm_ctas += m.parts;
    m.end_p = b.norm_ctas;
    b.tiles += static_cast<int>(xt);
    m.end_t = b.tiles;
    m.x0 = h.x[0];
    m.xn = h.x[a.steps & 1];
  }
  b.end = i;
  b.shapes.n = b.mats.n = i - at;
  b.mats.mu = a.mu;
  b.mats.eps = a.eps;
  b.mats.nesterov = a.nesterov;
  b.mats.update = a.update;
  const size_t tiles = static_cast<size_t>(used) * kTile;
  b.mats.partial = reinterpret_cast<double*>(tiles);  // an offset until the base is known
  b.bytes = tiles + static_cast<size_t>(partials) * sizeof(double);
  int tiles_a = 0, tiles_x = 0;
  if (exact) count_tiles<2, true>(b.shapes, tiles_a, tiles_x);
  else count_tiles<2, false>(b.shapes, tiles_a, tiles_x);
  b.pairs = tiles_x >= kPairTiles;
  if (exact) b.pairs ? plan_parts<2, true>(b) : plan_parts<1, true>(b);
  else b.pairs ? plan_parts<2, false>(b) : plan_parts<1, false>(b);
  return b;
}

#define ORTHO_RUN(...)                      \
  do {                                      \
    const cudaError_t e_ = (__VA_ARGS__);   \
    if (e_ != cudaSuccess) return e_;       \
  } while (0)

template <int CG, bool EXACT>
cudaError_t run_products(const sparge_ortho& a, Batch& b, uint8_t* ws, cudaStream_t st) {
  using C = GemmCfg<CG, EXACT>;
  CUtensorMap tm128, tm64;
  const int64_t bytes = reinterpret_cast<uint8_t*>(b.mats.partial) - ws;
  if (make_tmap_rows(&tm128, ws, bytes, 128) != 0 || make_tmap_rows(&tm64, ws, bytes, 64) != 0)
    return cudaErrorInvalidValue;
  auto grid = [](int items) { return CG * std::min(items, kSMs / CG); };
  const int grid_g = grid(b.items_g), grid_a = grid(b.tiles_a), grid_x = grid(b.tiles_x);
  GemmParams p = {ws, reinterpret_cast<float*>(ws + b.sums), b.mats.counts, 0, 0, a.a, a.b, a.c,
                  a.status};
  for (int i = 0; i < a.steps; ++i) {
    p.from = i & 1;
    p.tiles = b.items_g;
    ORTHO_RUN(launch_chained(ortho_gemm_kernel<CG, EXACT, kGram>, grid_g, C::kThreads, C::bytes, CG,
                             st, tm128, tm64, b.shapes, p));
    p.tiles = b.tiles_a;
    ORTHO_RUN(launch_chained(ortho_gemm_kernel<CG, EXACT, kSquare>, grid_a, C::kThreads, C::bytes, CG,
                             st, tm128, tm64, b.shapes, p));
    p.tiles = b.tiles_x;
    ORTHO_RUN(launch_chained(ortho_gemm_kernel<CG, EXACT, kApply>, grid_x, C::kThreads, C::bytes, CG,
                             st, tm128, tm64, b.shapes, p));
  }
  return cudaSuccess;
}

template <bool EXACT>
cudaError_t run_batch(const sparge_ortho& a, Batch& b, uint8_t* ws, cudaStream_t st) {
  b.mats.base = ws;
  b.mats.partial = reinterpret_cast<double*>(ws + reinterpret_cast<uintptr_t>(b.mats.partial));
  b.mats.counts = reinterpret_cast<int*>(ws + reinterpret_cast<uintptr_t>(b.mats.counts));
  ORTHO_RUN(launch_chained(ortho_norm_kernel, b.norm_ctas, 256, 0, 1, st, b.mats));
  ORTHO_RUN(launch_chained(ortho_start_kernel<EXACT>, std::min(b.tiles, kStartCtas), 256, 0, 1, st, b.mats));
  if (b.pairs)
    ORTHO_RUN(run_products<2, EXACT>(a, b, ws, st));
  else
    ORTHO_RUN(run_products<1, EXACT>(a, b, ws, st));
  ORTHO_RUN(launch_chained(ortho_finish_kernel<EXACT>, b.tiles, 256, 0, 1, st, b.mats));
  return cudaSuccess;
}
#undef ORTHO_RUN

#define ORTHO_TRY(expr)               \
  do {                                \
    const int rc_ = (expr);           \
    if (rc_ != SPARGE_OK) return rc_; \
  } while (0)

constexpr int kMaxSide = 65536, kMaxSteps = 64;

int check_sizes(const sparge_ortho* a) {
  if (a == nullptr || a->n < 1 || a->mats == nullptr) return SPARGE_ERR_INVALID_ARG;
  if (a->n > SPARGE_MAX_TENSORS) return SPARGE_ERR_UNSUPPORTED;
  for (int i = 0; i < a->n; ++i) {
    const sparge_matrix& m = a->mats[i];
    if (m.rows < 1 || m.cols < 1) return SPARGE_ERR_INVALID_ARG;
    if (m.rows > kMaxSide || m.cols > kMaxSide) return SPARGE_ERR_UNSUPPORTED;
  }
  return SPARGE_OK;
}

int check_place(const void* p, int64_t stride, int type, const sparge_matrix& m) {
  if (p == nullptr) return SPARGE_ERR_INVALID_ARG;
  if (type != SPARGE_BF16 && type != SPARGE_F32) return SPARGE_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(p) % (type == SPARGE_F32 ? 4 : 2) != 0) return SPARGE_ERR_MISALIGNED;
  if (m.rows > 1 && (stride < 1 || stride > int64_t(1) << 40)) return SPARGE_ERR_INVALID_ARG;
  return SPARGE_OK;
}

// A tensor of the list and what is done with it.
struct Place {
  Layout at;
  int mat;
  bool written, momentum;
};

int check_ortho(const sparge_ortho* a) {
  ORTHO_TRY(check_sizes(a));
  if (a->steps < 0 || a->steps > kMaxSteps) return SPARGE_ERR_INVALID_ARG;
  for (float f : {a->a, a->b, a->c})
    if (!(fabsf(f) <= 16.f)) return SPARGE_ERR_INVALID_ARG;
  if (!isfinite(a->eps) || a->eps < 0.f || !isfinite(a->mu)) return SPARGE_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(a->status) % 4 != 0) return SPARGE_ERR_MISALIGNED;
  std::vector<Place> places;
  places.reserve(3 * static_cast<size_t>(a->n));
  for (int i = 0; i < a->n; ++i) {
    const sparge_matrix& m = a->mats[i];
    ORTHO_TRY(check_place(m.grad, m.grad_stride, m.grad_type, m));
    ORTHO_TRY(check_place(m.out, m.out_stride, m.out_type, m));
    if (!isfinite(m.keep) || !isfinite(m.step)) return SPARGE_ERR_INVALID_ARG;
    auto put = [&](const void* p, int64_t stride, int type, bool written, bool momentum) {
      const int64_t size = type == SPARGE_F32 ? 4 : 2;
      places.push_back({layout_of(p, {m.rows, 1, 1}, {stride, 0, 0}, m.cols * size, size), i, written,
                        momentum});
    };
    put(m.grad, m.grad_stride, m.grad_type, false, false);
    put(m.out, m.out_stride, m.out_type, true, false);
    if (m.momentum != nullptr) {
      ORTHO_TRY(check_place(m.momentum, m.momentum_stride, SPARGE_F32, m));
      put(m.momentum, m.momentum_stride, SPARGE_F32, true, true);
    }
  }
  // In the order of their first bytes, each is compared with those before it that
  // reach so far.
  std::sort(places.begin(), places.end(),
            [](const Place& x, const Place& y) { return x.at.at < y.at.at; });
  std::vector<int> open;
  for (size_t i = 0; i < places.size(); ++i) {
    const Place& x = places[i];
    if (x.written && meets_itself(x.at)) return SPARGE_ERR_INVALID_ARG;
    size_t kept = 0;
    for (size_t k = 0; k < open.size(); ++k) {
      const Place& y = places[open[k]];
      if (y.at.span >= 0 && y.at.at + y.at.span <= x.at.at) continue;
      open[kept++] = open[k];
      if (!x.written && !y.written) continue;
      // (a result in its own gradient's place)
      if (x.mat == y.mat && x.written != y.written && !x.momentum && !y.momentum &&
          same_place(x.at, y.at) && !a->update)
        continue;
      if (meet(x.at, y.at)) return SPARGE_ERR_INVALID_ARG;
    }
    open.resize(kept);
    open.push_back(static_cast<int>(i));
  }
  return SPARGE_OK;
}

size_t workspace_of(const sparge_ortho& a) {
  size_t most = 0;
  for (int at = 0; at < a.n;) {
    const Batch b = make_batch(a, at);
    most = std::max(most, b.bytes);
    at = b.end;
  }
  return most;
}

}  // namespace

}  // namespace sparge

using namespace sparge;

extern "C" {

int sparge_orthogonalize_workspace_bytes(const sparge_ortho* args, size_t* bytes) {
  if (bytes == nullptr) return SPARGE_ERR_INVALID_ARG;
  ORTHO_TRY(check_sizes(args));
  *bytes = workspace_of(*args);
  return SPARGE_OK;
}

int sparge_orthogonalize_check(const sparge_ortho* args) try {
  return check_ortho(args);
} catch (...) {  // no memory for the list on the host
  return SPARGE_ERR_INVALID_ARG;
}

int sparge_orthogonalize(const sparge_ortho* args, void* workspace, size_t ws_bytes,
                         sparge_stream_t stream) try {
  ORTHO_TRY(check_ortho(args));
  if (workspace == nullptr || ws_bytes < workspace_of(*args)) return SPARGE_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) % 16 != 0) return SPARGE_ERR_MISALIGNED;
  for (int at = 0; at < args->n;) {
    Batch b = make_batch(*args, at);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const cudaError_t e = args->half ? run_batch<false>(*args, b, ws, stream)
                                     : run_batch<true>(*args, b, ws, stream);
    if (e != cudaSuccess) return SPARGE_ERR_CUDA;
    at = b.end;
  }
  return SPARGE_OK;
} catch (...) {  // no memory for the list on the host
  return SPARGE_ERR_INVALID_ARG;
}

}  // extern "C"
