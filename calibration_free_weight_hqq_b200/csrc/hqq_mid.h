// hqq_mid.h - tile sizes, shared memory and the division of work of the products of some tokens
// (hqq_mid_impl.cuh).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "hqq_kernels.h"
#include "hqq_tiles.h"

namespace hqqk {

constexpr int kMidRows = 128;    // output features per tile: the M of the MMA
constexpr int kMidLine = 64;     // contraction per 128-byte swizzled line
constexpr int kMidTokens = 256;  // tokens per tile at most: the N of the MMA
constexpr int kMidDqWarps = 16;  // two groups of 8 warps, alternate stages
constexpr int kMidEpiWarps = 4;
constexpr int kMidThreads = 32 * (2 + kMidDqWarps + kMidEpiWarps);
constexpr uint32_t kMidTileBytes = kMidRows * kMidLine * 2;  // a 128 x 64 tile of W'
constexpr int kMidMaxSmem = 232448;  // dynamic shared memory of a CTA at most: all of an SM's 227 KB
constexpr int64_t kMidMaxCols = int64_t(1) << 24;  // 32-bit offsets inside a tile's 128 rows

enum MidMode : int { kMidLinear = 0, kMidGated = 1, kMidBackward = 2 };

// Bytes of a warp's codes of a stage, and stages whose codes are in flight: 32 KB of them a CTA, 8 at
// most.
__host__ __device__ constexpr int mid_codes(int nbits, int mode) {
  return mode == kMidGated ? 2 * tile_bytes(nbits, 64) : tile_bytes(nbits, 128);
}
__host__ __device__ constexpr int mid_depth(int nbits, int mode) {
  const int n = 32768 / (kMidDqWarps * mid_codes(nbits, mode));
  return n < 1 ? 1 : n > 8 ? 8 : n;
}

// Contraction per k-block, a stage: two W' tiles each, of consecutive lines or, in the gated form, of
// gate and up. (Stages of one tile left the warp that issues the MMAs as the pace: its wait and
// commit cost some 700 cycles a stage at any token count.)
__host__ __device__ constexpr int mid_bk(int mode) { return mode == kMidGated ? 64 : 128; }

// What the host and the device need to agree on. A unit is one k-block of one tile (of both
// weights in the gated form); the units of all tiles, in order, are dealt out evenly to the
// CTAs, and a tile that several CTAs share is summed from their partial tiles.
struct MidPlan {
  int tok;             // tokens per tile, a multiple of 16
  int tok_tiles, row_tiles;
  int kb1, kb;         // k-blocks of one source, of a tile
  int ctas;
  int stages;
  uint32_t off_ring, off_bar, smem;
  size_t partial_bytes;
};

struct MidJob {
  int mode;
  const void* X[2];  // tokens x contraction; the second of two sources in kMidBackward
  WeightView w[2];
  int weights;       // 1 or 2
  int64_t M, rows, cols;  // tokens; the weights' shape
  int x_dtype;
  int nbits, group_size, meta_dtype, meta_group_size;
  int act;
  void *Y, *G, *U;   // outputs (kMidBackward: Y is dX)
  void* workspace;   // MidPlan::partial_bytes
};

// Whether the kernel takes a job of these sizes, and its plan.
bool mid_plan(const MidJob& job, MidPlan* plan);
cudaError_t launch_mid(const MidJob& job, cudaStream_t stream);
cudaError_t read_mid_timeouts(unsigned int* out);

}  // namespace hqqk
