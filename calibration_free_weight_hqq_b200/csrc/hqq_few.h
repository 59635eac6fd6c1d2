// hqq_few.h - tile sizes and shared memory of the few-token products (hqq_few_impl.cuh), and which
// jobs they take.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "hqq_kernels.h"
#include "hqq_tiles.h"

namespace hqqk {

constexpr int kFewTokens = 8;     // tokens of a launch: the N of the warp-level MMA
constexpr int64_t kFewMaxCols = int64_t(1) << 26;
constexpr int kFewRows = 16;      // weight rows per tile
constexpr int kFewKB = 256;       // codes of a row per k-block, two chunks of 32 for each of 4 lanes
constexpr int kFewMaxWarps = 16;  // warps of a CTA: 8 (two CTAs an SM) or 16
constexpr int kFewRedStride = kFewRows + 4;  // floats per token of a partial tile: the stores
                                             // of a fragment fall on 32 different banks
constexpr int kFewMaxSmem = 226 * 1024;  // dynamic shared memory of a CTA at most
constexpr int kFewRed = 8 * kFewRedStride * 4;  // bytes of one warp's partial tile

// k-blocks whose codes are in flight per warp: about 6 KB of them, 96 KB an SM at 16 warps (the
// memory's latency at full bandwidth asks for about 40), but 1 at least and 4 at most.
__host__ __device__ constexpr int few_depth(int nbits, int mats) {
  const int n = 6144 / (mats * tile_bytes(nbits, kFewKB));
  return n < 1 ? 1 : n > 4 ? 4 : n;
}
// Bytes of a token's row of X in shared memory (padded by 64).
__host__ __device__ constexpr uint32_t few_x_row(uint32_t K) {
  return (K + kFewKB - 1) / kFewKB * (2 * kFewKB) + 64;
}
// Dynamic shared memory of a CTA: X [tokens][k-blocks][256], partial tiles, code rings.
__host__ __device__ constexpr size_t few_smem(int nbits, int mats, int warps, int64_t M, int64_t K) {
  return static_cast<size_t>(M) * few_x_row(static_cast<uint32_t>(K)) +
         static_cast<size_t>(warps * mats) *
             (kFewRed + few_depth(nbits, mats) * tile_bytes(nbits, kFewKB));
}

// Warps of a CTA: 8 with two CTAs an SM where their X fits in half the shared memory (a CTA's
// barriers then pass under the other's work: 4 bits, 1 token, 11008 x 4096, 11.3 us against 12.7 with
// 16 warps, gated 21.1 against 23.6, 28672 x 8192 45.8 against 49.7; equal at 8 tokens), else 16; 0
// where X does not fit at all, or the row length exceeds the kernel's 32-bit offsets inside a tile, or
// there are more tokens than an MMA takes. (The some-token kernel is slower wherever this one serves at full speed:
// 11008 x 4096, 8 tokens here 14 us, 24 tokens there 21.5, and its time hardly depends on tokens there.)
inline int few_warps(const FewJob& j) {
  if (j.M > kFewTokens || j.K > kFewMaxCols) return 0;
  if (few_smem(j.nbits, j.mats, 8, j.M, j.K) <= 113 * 1024) return 8;
  return few_smem(j.nbits, j.mats, 16, j.M, j.K) <= kFewMaxSmem ? 16 : 0;
}

}  // namespace hqqk
