// hqq_few_impl.cuh - products of up to 8 tokens with quantized weights of any format (axis 1).
//
// Y[m, n] = dt( sum_k X[m, k] W'[n, k] + bias[n] ), W' = dt((code - zero) * scale) exactly as the
// dequantizer writes it, fp32 accumulation; with two weights (the gated pair)
// Y = dt( act(X Wg'^T + bg) * (X Wu'^T + bu) ), both projections in one pass.
//
// With so few tokens the packed weight is read once and the work is its conversion. Each warp
// converts codes in registers straight into the A fragments of the warp-level MMA
// (mma.sync m16n8k16, fp32 accumulators): 16 weight rows are its M, the tokens its N, and
// W' passes through no memory.
//   * k-blocks of 256: lane (g, t) = (lane / 4, lane % 4) takes the 64 consecutive codes
//     k = 64t .. 64t+63 of rows g and g + 8, in two chunks of 32, and of X the same 64 values of
//     token g. An MMA's k slots {2t, 2t+1, 2t+8, 2t+9} are lane t's own, so which codes sit there is
//     free as long as X agrees: the order is the one in which masks take codes out of their words.
//   * X stays in shared memory for the kernel's life, its 16-byte pieces reordered so that a
//     warp's reads are free of bank conflicts. CTAs are persistent over tiles of 16 rows.
//   * The warps of a CTA split K, k-block by k-block in turn; their partial sums meet in shared
//     memory and are added in warp order (deterministic).
//   * Codes come by asynchronous copies a few k-blocks ahead (across tiles too), each warp its own;
//     scale and zero one k-block ahead in registers.
//   * Lanes without a token of their own (g >= M) repeat the last one; those results are dropped.
// What bounds it: instructions (4.35 a code and lane at 4 bits and 1 token, 7.8 at 3 bits with 8-bit meta and
// 5 tokens), then their latency: at 16 warps an SM (the registers hold no more) 49 and 67 % of the issue
// slots are taken. Measured, group 64: 11008 x 4096, 4 bits, 1
// token 11 us (2.3 TB/s; its bytes take 3.9 us at a copy's rate), the gated pair 21 us; 28672 x 8192, 4
// bits, 1 token 46 us (2.9 TB/s), 3 bits with 8-bit scale and zero, 5 tokens 86 us.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "hqq_act.cuh"
#include "hqq_codes.cuh"
#include "hqq_device.cuh"
#include "hqq_few.h"
#include "hqq_kernels.h"
#include "hqq_tensor.cuh"

namespace hqqk {
namespace {

struct FewArgs {
  WeightArgs w;
  const uint8_t* X;
  unsigned short *Y, *G, *U;
  int M, N, K;
  int act;
};

// One chunk of rows g and g + 8 as A fragments against X's as B, units alternating between two
// accumulators (each MMA waits for the one before it on the same registers). m0, m1: the chunk's
// GROUPS groups in the two rows.
template <int NBITS, bool F16, int GROUPS, bool ONE>
__device__ __forceinline__ void multiply_chunk(float (&acc)[2][4], const Codes32<NBITS> (&c)[2],
                                               const GroupMeta* m0, const GroupMeta* m1,
                                               const uint4* x) {
  constexpr int OUT = F16 ? kF16 : kBF16;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const uint4 xu = x[4 * u];
    const uint4 w0 = dequant_unit<NBITS, OUT, GROUPS, ONE>(c[0], u, m0);
    const uint4 w1 = dequant_unit<NBITS, OUT, GROUPS, ONE>(c[1], u, m1);
    mma_16816<F16>(acc[u & 1], w0.x, w1.x, w0.y, w1.y, xu.x, xu.y);
    mma_16816<F16>(acc[u & 1], w0.z, w1.z, w0.w, w1.w, xu.z, xu.w);
  }
}

// X [M][K] into shared memory, [M][KB][32 pieces of 8 values]: unit p (0 .. 7) of lane t's two chunks,
// in slot_element's order, at piece 4p + t. Rows are padded by four pieces, so that 8 lanes - two
// tokens, four t - read 8 different pieces mod 8.
template <int NBITS>
__device__ __forceinline__ void stage_x(uint4* xs, const uint8_t* X, uint32_t M, uint32_t K,
                                        uint32_t KB) {
  const uint32_t chunks = KB * 8;  // of 32 values
  for (uint32_t i = threadIdx.x; i < M * chunks; i += blockDim.x) {
    const uint32_t tok = i / chunks, c = i - tok * chunks;
    const uint8_t* src = X + (static_cast<int64_t>(tok) * K + c * 32) * 2;
    uint32_t v[16];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (c * 32 + 8 * q < K) w = __ldg(reinterpret_cast<const uint4*>(src) + q);
      v[4 * q] = w.x;
      v[4 * q + 1] = w.y;
      v[4 * q + 2] = w.z;
      v[4 * q + 3] = w.w;
    }
    uint4* dst = xs + tok * (KB * 32 + 4) + (c / 8) * 32 + 16 * (c & 1) + ((c & 7) >> 1);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      uint32_t o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int a = slot_element<NBITS>(u, 2 * q), b = slot_element<NBITS>(u, 2 * q + 1);
        o[q] = __byte_perm(v[a / 2], v[b / 2], (a % 2 ? 0x32 : 0x10) | (b % 2 ? 0x7600 : 0x5400));
      }
      dst[4 * u] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// GROUP: 64 (groups of 64 codes or more), 32, 16 (whole_rows) or 8 (any group size and K; codes and
// meta read where they are used). ANY: see RawMeta.
template <int NBITS, bool F16, int MATS, int GROUP, bool ANY>
__global__ void __launch_bounds__(32 * kFewMaxWarps, 1) few_tokens_kernel(const FewArgs a) {
  constexpr int OUT = F16 ? kF16 : kBF16;
  constexpr bool kWhole = GROUP != 8;
  constexpr int kGroups = 64 / GROUP;            // groups of a lane's codes of a k-block
  constexpr int kGroupsHalf = kGroups > 1 ? kGroups / 2 : 1;
  constexpr bool kTwos = GROUP == 16 && !ANY;    // meta by two groups
  constexpr int kDepth = few_depth(NBITS, MATS);
  using Tile = CodeTile<NBITS, kFewKB, true>;
  constexpr int kTile = tile_bytes(NBITS, kFewKB);  // a warp's k-block
  extern __shared__ __align__(16) uint8_t smem[];
  // the shuffle tells the compiler that a warp's index, and all that follows from it, is uniform
  const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);
  const uint32_t warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  const uint32_t g = lane >> 2, t = lane & 3;
  const uint32_t K = static_cast<uint32_t>(a.K), KB = (K + kFewKB - 1) / kFewKB;
  const uint32_t groups_per_row = K >> a.w.lg_group;
  const uint32_t tiles = (static_cast<uint32_t>(a.N) + kFewRows - 1) / kFewRows;
  uint4* xs = reinterpret_cast<uint4*>(smem);
  uint8_t* after_x = smem + static_cast<size_t>(a.M) * few_x_row(K);
  float* red = reinterpret_cast<float*>(after_x);  // [MATS][warps][8][kFewRedStride]
  uint8_t* ring = after_x + MATS * warps * kFewRed + warp * (kDepth * MATS * kTile);
  const uint32_t ring_u = smem_u32(ring);

  // Rows g and g + 8 of a tile. N is a multiple of 8: rows 8 .. 15 all exist or none does, and where
  // they do not (the last tile), rows 0 .. 7 are read in their place and the results dropped.
  auto second_row = [&](uint32_t tile) {
    return tile * kFewRows + 8 < static_cast<uint32_t>(a.N) ? g + 8 : g;
  };
  auto make_slab = [&](int i, uint32_t tile) {
    return slab_of_row<NBITS, ANY>(a.w, i, static_cast<int64_t>(tile) * kFewRows, K, groups_per_row);
  };

  // --- codes, kDepth k-blocks ahead: (copy_tile, copy_kb) is the next to ask for
  constexpr uint32_t kStepCodes = NBITS == 3 ? kFewKB : kFewKB / 8 * NBITS;
  const uint32_t row_step = NBITS == 3 ? K : K / 8 * NBITS;
  uint32_t copy_tile = warp < KB ? blockIdx.x : tiles, copy_kb = warp;
  const uint8_t* copy_base[MATS];
  uint32_t copy_code0[MATS];
  auto aim_copies = [&]() {
    if (copy_tile < tiles) {
#pragma unroll
      for (int i = 0; i < MATS; ++i) {
        const Slab b = make_slab(i, copy_tile);
        copy_base[i] = b.codes;
        copy_code0[i] = b.code0;
      }
    }
  };
  auto copy_next = [&](uint32_t st) {
    if (copy_tile < tiles) {
      const uint32_t rows = min(static_cast<uint32_t>(kFewRows),
                                static_cast<uint32_t>(a.N) - copy_tile * kFewRows);
      const uint32_t codes = min(static_cast<uint32_t>(kFewKB), K - copy_kb * kFewKB);
#pragma unroll
      for (int i = 0; i < MATS; ++i) {
        const uint32_t to = ring_u + (st * MATS + i) * kTile, step = copy_kb * kStepCodes;
        Tile::copy(to, copy_base[i] + (NBITS == 3 ? 0u : step), copy_code0[i] + step, row_step, rows,
                   codes, lane);
      }
      copy_kb += warps;
      if (copy_kb >= KB) {
        copy_kb = warp;
        copy_tile += gridDim.x;
        aim_copies();
      }
    }
    cp_async_commit();
  };
  if constexpr (kWhole) {
    aim_copies();
#pragma unroll 1
    for (uint32_t s = 0; s < kDepth; ++s) copy_next(s);
  }

  stage_x<NBITS>(xs, a.X, static_cast<uint32_t>(a.M), K, KB);
  __syncthreads();
  const uint4* xrow = xs + min(g, static_cast<uint32_t>(a.M) - 1) * (few_x_row(K) / 16) + t;

  // --- scale and zero, one k-block ahead. A k-block is a whole number of groups, so a lane's place
  // in a tile and a k-block's (uniform) add up here too.
  Slab slab[MATS];
  uint32_t row1 = g;
  uint32_t meta_at[2] = {g * groups_per_row + ((64 * t) >> a.w.lg_group), 0};
  RawMeta<ANY> next[MATS][2][kGroups];
  auto aim = [&](uint32_t tile) {
#pragma unroll
    for (int i = 0; i < MATS; ++i) slab[i] = make_slab(i, tile);
    row1 = second_row(tile);
    meta_at[1] = row1 * groups_per_row + ((64 * t) >> a.w.lg_group);
  };
  auto fetch_meta = [&](uint32_t kb) {
    const uint32_t step = (kb * kFewKB) >> a.w.lg_group;
    const bool whole = (kb + 1) * kFewKB <= K;
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
      if (!whole && kb * kFewKB + 64 * t + GROUP * u >= K) break;
#pragma unroll
      for (int i = 0; i < MATS; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if constexpr (!kTwos)
            next[i][r][u] = load_raw_meta<ANY>(slab[i], a.w, step, meta_at[r] + u);
          else if (u % 2 == 0)
            next[i][r][u] = load_raw_meta_two(slab[i], step, meta_at[r] + u);
        }
    }
  };
  if (warp < KB && blockIdx.x < tiles) {
    aim(blockIdx.x);
    if constexpr (kWhole) fetch_meta(warp);
  }

  uint32_t st = 0;
  for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    float acc[MATS][2][4];
#pragma unroll
    for (int i = 0; i < MATS; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][h][q] = 0.0f;
#pragma unroll 1
    for (uint32_t kb = warp; kb < KB; kb += warps) {
      const uint4* x = xrow + kb * 32;
      if constexpr (kWhole) {
        const bool tail = (kb + 1) * kFewKB > K;
        GroupMeta m[MATS][2][kGroups];
        Exactness known;
#pragma unroll
        for (int i = 0; i < MATS; ++i)
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int u = 0; u < kGroups; ++u) {
              RawMeta<ANY> raw = next[i][r][u];
              if constexpr (kTwos) raw = one_of_two(next[i][r][u & ~1], u % 2);
              float2 sz = meta_f32_pair<ANY, F16>(raw, slab[i], a.w.meta_dt);
              if (tail && kb * kFewKB + 64 * t + GROUP * u >= K)
                sz = make_float2(0.0f, 0.0f);  // W' = 0 past K
              m[i][r][u] = group_meta<NBITS, F16>(sz.x, sz.y, &known);
            }
        const bool one = !ANY && __all_sync(0xFFFFFFFFu, known.holds());
        uint32_t slot[MATS][2];  // 3 bits: the first code's place in its 16 bytes, of both rows
#pragma unroll
        for (int i = 0; i < MATS; ++i) {
          slot[i][0] = slot[i][1] = 0u;
          if constexpr (NBITS == 3) {
            slot[i][0] = (slab[i].code0 + g * K + kb * kFewKB) % 40u;
            slot[i][1] = (slab[i].code0 + (g + 8) * K + kb * kFewKB) % 40u;
          }
        }
        // the next k-block's meta, of the next tile after this one's last
        if (kb + warps < KB) {
          fetch_meta(kb + warps);
        } else if (tile + gridDim.x < tiles) {
          aim(tile + gridDim.x);
          fetch_meta(warp);
        }
        const uint8_t* block = ring + st * (MATS * kTile);
        cp_async_wait<kDepth - 1>();
        __syncwarp();  // every lane's copies have landed
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int i = 0; i < MATS; ++i) {
            Codes32<NBITS> c[2];
#pragma unroll
            for (int r = 0; r < 2; ++r)
              c[r] = Tile::read(block + i * kTile, g + 8 * r, 64 * t + 32 * h, slot[i][r]);
            const GroupMeta* m0 = m[i][0] + (kGroups > 1 ? h * kGroupsHalf : 0);
            const GroupMeta* m1 = m[i][1] + (kGroups > 1 ? h * kGroupsHalf : 0);
            if (one)
              multiply_chunk<NBITS, F16, kGroupsHalf, true>(acc[i], c, m0, m1, x + 16 * h);
            else
              multiply_chunk<NBITS, F16, kGroupsHalf, false>(acc[i], c, m0, m1, x + 16 * h);
          }
        }
        __syncwarp();  // every lane has read them
        copy_next(st);
        st = st + 1 == kDepth ? 0 : st + 1;
      } else {
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const uint32_t kh = kb * kFewKB + 64 * t + 32 * h;
          const int units = kh < K ? static_cast<int>(min(4u, (K - kh) / 8)) : 0;
#pragma unroll
          for (int i = 0; i < MATS; ++i) {
            Codes32<NBITS> c[2];
            GroupMeta m[2][4];
            Exactness known;  // not used
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint32_t row = r == 0 ? g : row1;
              c[r] = load_codes_units<NBITS>(slab[i].codes, slab[i].code0 + row * K + kh, units);
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                float2 sz = make_float2(0.0f, 0.0f);
                if (u < units)
                  sz = meta_f32_pair<ANY, F16>(
                      load_raw_meta<ANY>(slab[i], a.w, 0u,
                                         row * groups_per_row + ((kh + 8 * u) >> a.w.lg_group)),
                      slab[i], a.w.meta_dt);
                m[r][u] = group_meta<NBITS, F16>(sz.x, sz.y, &known);
              }
            }
            multiply_chunk<NBITS, F16, 4, false>(acc[i], c, m[0], m[1], x + 16 * h);
          }
        }
        if (kb + warps >= KB && tile + gridDim.x < tiles) aim(tile + gridDim.x);
      }
    }

#pragma unroll
    for (int i = 0; i < MATS; ++i) {
      float* p = red + (i * warps + warp) * (8 * kFewRedStride) + 2 * t * kFewRedStride + g;
      p[0] = __fadd_rn(acc[i][0][0], acc[i][1][0]);
      p[kFewRedStride] = __fadd_rn(acc[i][0][1], acc[i][1][1]);
      p[8] = __fadd_rn(acc[i][0][2], acc[i][1][2]);
      p[kFewRedStride + 8] = __fadd_rn(acc[i][0][3], acc[i][1][3]);
    }
    __syncthreads();
    const int row = threadIdx.x % kFewRows, m = threadIdx.x / kFewRows;
    const int64_t n = static_cast<int64_t>(tile) * kFewRows + row;
    if (m < a.M && n < a.N) {
      float v[MATS];
#pragma unroll
      for (int i = 0; i < MATS; ++i) {
        v[i] = 0.0f;
        for (uint32_t w = 0; w < warps; ++w)
          v[i] = __fadd_rn(v[i], red[(i * warps + w) * (8 * kFewRedStride) + m * kFewRedStride + row]);
        if (a.w.bias[i] != nullptr) {
          const uint32_t b = a.w.bias[i][n];
          v[i] = __fadd_rn(v[i], F16 ? f16_bits_to_f32(b) : bf16_bits_to_f32(b));
        }
      }
      const int64_t at = static_cast<int64_t>(m) * a.N + n;
      auto bits = [](float f) { return static_cast<unsigned short>(pack2_16<OUT>(f, 0.0f)); };
      if constexpr (MATS == 2) {
        if (a.G != nullptr) a.G[at] = bits(v[0]);
        if (a.U != nullptr) a.U[at] = bits(v[1]);
        const float h = a.act == kSilu   ? act_f32<kSilu>(v[0])
                        : a.act == kGelu ? act_f32<kGelu>(v[0])
                                         : act_f32<kGeluTanh>(v[0]);
        a.Y[at] = bits(__fmul_rn(h, v[1]));
      } else {
        a.Y[at] = bits(v[0]);
      }
    }
    __syncthreads();  // the partial tiles are free again
  }
}

template <int NBITS, bool F16, int MATS>
cudaError_t launch_few_typed(const FewJob& j, const FewArgs& a, cudaStream_t st) {
  const int warps = few_warps(j);
  if (warps == 0) return cudaErrorInvalidValue;
  const int64_t tiles = (j.N + kFewRows - 1) / kFewRows;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(tiles, kSms * (16 / warps)));
  const size_t smem = few_smem(NBITS, MATS, warps, j.M, j.K);
  const bool any = any_meta(j.w, j.mats, j.meta_dtype, j.x_dtype);
  auto kernel = few_tokens_kernel<NBITS, F16, MATS, 8, true>;
  if (whole_rows(NBITS, j.K)) {
    if (j.group_size >= 64)
      kernel = any ? few_tokens_kernel<NBITS, F16, MATS, 64, true>
                   : few_tokens_kernel<NBITS, F16, MATS, 64, false>;
    else if (j.group_size == 32)
      kernel = any ? few_tokens_kernel<NBITS, F16, MATS, 32, true>
                   : few_tokens_kernel<NBITS, F16, MATS, 32, false>;
    else if (j.group_size == 16 && !any && meta_by_twos(j.w, j.mats))
      kernel = few_tokens_kernel<NBITS, F16, MATS, 16, false>;
    else if constexpr (MATS == 1) {
      // 2 bits, 8-bit meta, 11008 x 4096, 1 token: 21 us against 35. A pair's meta, eight groups of
      // two weights ahead, does not fit the registers (90 us against 84).
      if (j.group_size == 16) kernel = few_tokens_kernel<NBITS, F16, MATS, 16, true>;
    }
  }
  if (smem > 48 * 1024) {
    // always the most, never this call's: a smaller value, set by another thread between here and the
    // launch, would have the launch refused
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewMaxSmem);
    if (e != cudaSuccess) return e;
  }
  kernel<<<grid, 32 * warps, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

// One weight (mats 1) or the gated pair (mats 2) at NBITS; see FewJob.
template <int NBITS>
cudaError_t launch_few_bits(const FewJob& j, cudaStream_t st) {
  FewArgs a = {};
  a.w = weight_args(j.w, j.mats, j.group_size, j.meta_dtype, j.meta_group_size);
  a.X = static_cast<const uint8_t*>(j.X);
  a.Y = static_cast<unsigned short*>(j.Y);
  a.G = static_cast<unsigned short*>(j.G);
  a.U = static_cast<unsigned short*>(j.U);
  a.M = static_cast<int>(j.M);
  a.N = static_cast<int>(j.N);
  a.K = static_cast<int>(j.K);
  a.act = j.act;
  const bool f16 = j.x_dtype == kF16;
  if (j.mats == 1)
    return f16 ? launch_few_typed<NBITS, true, 1>(j, a, st)
               : launch_few_typed<NBITS, false, 1>(j, a, st);
  return f16 ? launch_few_typed<NBITS, true, 2>(j, a, st)
             : launch_few_typed<NBITS, false, 2>(j, a, st);
}

}  // namespace hqqk
