// What the kernels of the attention over a context share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "sparge.h"

namespace sparge {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kCrossQ = 128;  // queries of a tile
constexpr int kCrossK = 128;  // keys of a tile of the backward

// A tensor [batch, heads, tokens, d] as the kernels index it: strides in elements.
struct HeadsView {
  void* p;
  int64_t sb, sh, sn;
};

// Geometry of a validated sparge_cross.
struct CrossGeom {
  int B, Bk, H, Hk, N, M, d;
  int group;   // query heads to a key head
  int Mq;      // query tiles of a head
  int Mt;      // key tiles of a head
  float scale;
  const int32_t* kv_len;
};

// Valid keys of sample b.
SPARGE_DEV int cross_len(const CrossGeom& g, int b) {
  return g.kv_len == nullptr ? g.M : min(max(__ldg(g.kv_len + b), 0), g.M);
}

// Zeros the rows [first, rows) of a 128-byte-swizzled tile in shared memory (whole
// rows, so the swizzle does not matter), for the MMAs that follow.  One warp.
SPARGE_DEV void zero_tile_rows(uint8_t* tile, int chunks, uint32_t chunk_bytes, int first, int rows,
                               int lane) {
  for (int c = 0; c < chunks; ++c)
    for (int i = first * 8 + lane; i < rows * 8; i += 32)
      reinterpret_cast<uint4*>(tile + c * chunk_bytes)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  __syncwarp();
}

// cross_fwd.cu: workspace, launch.
size_t cross_fwd_workspace_bytes(const CrossGeom& g);
cudaError_t launch_cross_fwd(const CrossGeom& g, const sparge_cross& a, void* workspace,
                             cudaStream_t st);
// cross_fwd_wide.cu: the form for query tiles that fill the machine (no workspace).
cudaError_t launch_cross_fwd_wide(const CrossGeom& g, const sparge_cross& a, cudaStream_t st);
// cross_bwd.cu
size_t cross_bwd_workspace_bytes(const CrossGeom& g);
cudaError_t launch_cross_bwd(const CrossGeom& g, const sparge_cross& a, void* workspace,
                             cudaStream_t st);

}  // namespace sparge
