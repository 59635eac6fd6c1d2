// hqq_mid_impl.cuh - products of some tokens (from 9 to some hundreds) straight from the codes (axis 1).
//
//   linear:   Y[m, n]  = dt( sum_k X[m, k] W'[n, k] + bias[n] )
//   gated:    Y[m, n]  = dt( act(X Wg'^T + bg) * (X Wu'^T + bu) )
//   backward: dX[m, k] = dt( sum over sources and n of dY[m, n] W'[n, k] )
//
// Too many tokens for the warp-level MMA of the few-token kernel and too few to pay for writing the
// dequantized weight to memory and reading it back: W' goes from the codes into shared memory and
// no further. The roles of the operands swap against the usual product: 128 output features are
// the M of tcgen05.mma and up to 256 tokens its N, so that any number of tokens uses whole MMAs.
//   * Two groups of 8 warps convert codes into the 128-byte-swizzled operand layout, alternate
//     stages of two 128 x 64 W' tiles (consecutive in k, or in the gated form of gate and up). A
//     thread converts 64 codes a stage. Backward the same bytes are an MN-major operand: the
//     contraction runs along the weight's rows, the features along its columns; nothing is
//     transposed.
//   * One warp loads X (TMA, same swizzle), one thread issues the MMAs into TMEM, four warps empty
//     finished accumulators while the next tile runs (two accumulators when TMEM holds them).
//   * Work: all tiles' k-blocks in one line, cut evenly over the CTAs. A CTA that has a tile's whole
//     contraction writes the result; partial tiles go to the workspace in fp32 and a second kernel
//     adds them in order (deterministic).
//   * Codes come by asynchronous copies some stages ahead, each warp its own 16 rows; scale and zero
//     one stage ahead in registers.
// What bounds it: the converting warps (48-68 % of the issue slots, the tensor core waits for them) and at
// 256 tokens, where two stages fit, the wait of one for the other. Measured, 4 bits, group 64, 11008 x 4096,
// one after another: 24 us at 64 tokens, 43 us at 256 (540 TFLOP/s), gated 44 and 77 us; gradient of 4096
// x 11008 25 and 44 us. Gate and up in one tile share X and meet in the epilogue.
// Every wait is bounded (about two seconds); on expiry the CTA raises an abort flag, counts the
// timeout, skips its remaining work, waits for its copies in flight and frees its TMEM. Its partial tiles are
// marked as missing, and outputs that need one are not written.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "hqq_act.cuh"
#include "hqq_codes.cuh"
#include "hqq_device.cuh"
#include "hqq_mid.h"
#include "hqq_tensor.cuh"

namespace hqqk {
namespace {

struct MidArgs {
  WeightArgs w;
  float* partial;  // [cta][2][weights of a tile][tokens][128]
  unsigned short *Y, *G, *U;
  int M, rows, cols, out;  // tokens; the weights' shape; output features
  int act;
  MidPlan p;
};

constexpr int kMidFull = 0, kMidEmpty = 4, kMidAccFull = 8, kMidAccEmpty = 10, kMidBars = 12;

// K-major, or MN-major (see the same in hqq_dense.cu: 64-column blocks 8 KB apart, 8-line atoms
// 1 KB apart along the contraction).
__device__ __forceinline__ uint64_t mid_mnmajor_desc(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(8192 >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// A CTA's units [first, last) of the line of all tiles' k-blocks.
__device__ __forceinline__ uint32_t mid_first_unit(uint32_t cta, uint32_t ctas, uint32_t units) {
  return static_cast<uint32_t>(static_cast<uint64_t>(cta) * units / ctas);
}
__device__ __forceinline__ uint32_t mid_cta_of(uint32_t unit, uint32_t ctas, uint32_t units) {
  return static_cast<uint32_t>(((static_cast<uint64_t>(unit) + 1) * ctas - 1) / units);
}

// One output of the gated pair or of a plain product: bias, activation, product, rounding.
template <bool F16, int MATS>
__device__ __forceinline__ void mid_store(const MidArgs& a, int64_t tok, int n, float g, float u) {
  constexpr int OUT = F16 ? kF16 : kBF16;
  auto bits = [](float f) { return static_cast<unsigned short>(pack2_16<OUT>(f, 0.0f)); };
  auto value = [](unsigned short b) { return F16 ? f16_bits_to_f32(b) : bf16_bits_to_f32(b); };
  if (a.w.bias[0] != nullptr) g = __fadd_rn(g, value(__ldg(a.w.bias[0] + n)));
  const int64_t at = tok * a.out + n;
  if constexpr (MATS == 2) {
    if (a.w.bias[1] != nullptr) u = __fadd_rn(u, value(__ldg(a.w.bias[1] + n)));
    if (a.G != nullptr) a.G[at] = bits(g);
    if (a.U != nullptr) a.U[at] = bits(u);
    const float h = a.act == kSilu   ? act_f32<kSilu>(g)
                    : a.act == kGelu ? act_f32<kGelu>(g)
                                     : act_f32<kGeluTanh>(g);
    a.Y[at] = bits(__fmul_rn(h, u));
  } else {
    a.Y[at] = bits(g);
  }
}

__device__ __forceinline__ void mid_tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11,"
      " %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// GROUP: 64 (groups of 64 codes or more), 32, 16 (whole_rows) or 8 (any group size and cols; codes and
// meta read where they are used). ANY: see RawMeta.
template <int NBITS, bool F16, int MODE, int GROUP, bool ANY>
__global__ void __launch_bounds__(kMidThreads, 1)
    mid_tokens_kernel(const __grid_constant__ CUtensorMap map_x0,
                      const __grid_constant__ CUtensorMap map_x1, const MidArgs a) {
  constexpr int OUT = F16 ? kF16 : kBF16;
  constexpr int MATS = MODE == kMidGated ? 2 : 1;
  constexpr bool kWhole = GROUP != 8;
  // A thread converts two chunks of 32 codes a stage: 64 in a row, or in the gated form 32 of either
  // weight. Their groups:
  constexpr int kGroups = GROUP >= 32 ? 1 : 32 / GROUP;
  constexpr bool kTwos = GROUP == 16 && !ANY;  // meta by two groups
  constexpr bool kShared = MODE != kMidGated && GROUP >= 64;  // both chunks lie in one group
  constexpr int kBK = mid_bk(MODE);
  constexpr int kDepth = mid_depth(NBITS, MODE);
  using Tile = CodeTile<NBITS, kBK, false>;
  constexpr int kTile = tile_bytes(NBITS, kBK);  // a warp's codes of a stage (of either weight)
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t T = static_cast<uint32_t>(a.p.tok), KB = static_cast<uint32_t>(a.p.kb);
  const uint32_t units = static_cast<uint32_t>(a.p.row_tiles * a.p.tok_tiles) * KB;
  const uint32_t first = mid_first_unit(blockIdx.x, gridDim.x, units);
  const uint32_t count = mid_first_unit(blockIdx.x + 1, gridDim.x, units) - first;
  const uint32_t stages = static_cast<uint32_t>(a.p.stages);
  const uint32_t line_x = T * (2 * kMidLine), stage_bytes = 2 * kMidTileBytes + T * (2 * kBK);
  const uint32_t bufs = 2 * MATS * T <= 512 ? 2 : 1;
  volatile uint32_t* abort_flag =
      reinterpret_cast<volatile uint32_t*>(smem + a.p.off_bar + 8 * kMidBars + 4);
  auto bar = [&](uint32_t i) { return sbase + a.p.off_bar + 8u * i; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < 4; ++s) {
      mbar_init(bar(kMidFull + s), kMidDqWarps / 2 + 1);  // the converting warps and the copy of X
      mbar_init(bar(kMidEmpty + s), 1);                   // the MMAs' commit
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(kMidAccFull + s), 1);
      mbar_init(bar(kMidAccEmpty + s), kMidEpiWarps);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     bar(kMidBars)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(
      0xFFFFFFFFu, *reinterpret_cast<volatile uint32_t*>(smem + a.p.off_bar + 8 * kMidBars), 0);

  // mid_finish_kernel may take its place now; it waits for this grid's end before it reads
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == 0) {
    // ------------------------------------------------------------ X producer
    uint32_t tile = first / KB, kb = first - tile * KB, pos = 0, s = 0, phase = 1;
    int m0 = static_cast<int>((tile % a.p.tok_tiles) * T);
    for (; pos < count; ++pos) {
      if (!mbar_wait_idle(bar(kMidEmpty + s), phase, abort_flag)) break;
      if (lane == 0) {
        const bool second = MODE == kMidBackward && kb >= static_cast<uint32_t>(a.p.kb1);
        const CUtensorMap* map = second ? &map_x1 : &map_x0;
        const int k = static_cast<int>(second ? kb - a.p.kb1 : kb) * kBK;
        const uint32_t dst = sbase + s * stage_bytes + 2 * kMidTileBytes;
        mbar_arrive_tx(bar(kMidFull + s), T * (2 * kBK));
        tma_load_2d(dst, map, k, m0, bar(kMidFull + s));
        if (kBK == 2 * kMidLine) tma_load_2d(dst + line_x, map, k + kMidLine, m0, bar(kMidFull + s));
      }
      __syncwarp();
      if (++kb == KB) {
        kb = 0;
        ++tile;
        m0 = static_cast<int>((tile % a.p.tok_tiles) * T);
      }
      if (++s == stages) {
        s = 0;
        phase ^= 1;
      }
    }
    if (lane == 0) {  // own copies landed before leaving (complete on the normal path)
      for (uint32_t n = 0; n < stages && n < pos; ++n) {
        const uint32_t j = pos - 1 - n;
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(bar(kMidFull + j % stages), (j / stages) & 1) &&
               globaltimer() - t0 < kWaitLimitNs) {
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks along, so that its counters and descriptors stay in uniform registers;
    // an elected lane issues. This loop's latency paces small token counts: ring positions and
    // phases are counted, not divided out, and a stage has one barrier each way.
    constexpr uint32_t fmt = F16 ? 0u : 1u;
    constexpr bool kMN = MODE == kMidBackward;
    const uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | (kMN ? 1u << 15 : 0u) |
                           ((T >> 3) << 17) | (static_cast<uint32_t>(kMidRows >> 4) << 24);
    const uint64_t desc_w = kMN ? mid_mnmajor_desc(sbase) : sw128_kmajor_desc(sbase);
    const uint64_t desc_x = sw128_kmajor_desc(sbase + 2 * kMidTileBytes);
    const uint32_t issue = elect_one();
    uint32_t kb = first % KB, s = 0, phase = 0, buf = 0, phase_acc = 1, pos = 0;
    bool begins = true;
    for (; pos < count; ++pos) {
      bool go = !begins || mbar_wait(bar(kMidAccEmpty + buf), phase_acc, abort_flag);
      go = go && mbar_wait(bar(kMidFull + s), phase, abort_flag);
      if (!__all_sync(0xFFFFFFFFu, go)) break;
      tc_fence_after();
      const uint64_t at = static_cast<uint64_t>(s * (stage_bytes >> 4));
      const uint32_t acc = tmem + buf * MATS * T;
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // the stage's two W' tiles, 16 of the contraction at a time
        const uint64_t dw = desc_w + at + h * (kMidTileBytes >> 4);
        const uint64_t dx = desc_x + at + (MATS == 2 ? 0 : h * static_cast<uint64_t>(line_x >> 4));
#pragma unroll
        for (int k = 0; k < kMidLine / 16; ++k)
          tc_mma_one(MATS == 2 ? acc + h * T : acc, dw + (kMN ? 128 : 2) * k, dx + 2 * k, idesc,
                     !begins || k != 0 || (MATS == 1 && h != 0), issue);
      }
      tc_commit_one(bar(kMidEmpty + s), issue);
      begins = ++kb == KB;
      if (begins) kb = 0;
      if (++s == stages) {
        s = 0;
        phase ^= 1;
      }
      if (begins || pos + 1 == count) {
        tc_commit_one(bar(kMidAccFull + buf), issue);
        if (++buf == bufs) {
          buf = 0;
          phase_acc ^= 1;
        }
      }
    }
    if (lane == 0) {  // the issued MMAs have read their operands before the CTA leaves
      for (uint32_t n = 0; n < stages && n < pos; ++n) {
        const uint32_t j = pos - 1 - n;
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(bar(kMidEmpty + j % stages), (j / stages) & 1) &&
               globaltimer() - t0 < kWaitLimitNs) {
        }
      }
    }
    __syncwarp();
  } else if (warp < 2 + kMidDqWarps) {
    // ------------------------------------------------------------ codes to W'
    const uint32_t group = (warp - 2) / 8, wi = (warp - 2) % 8;
    const uint32_t rows = static_cast<uint32_t>(a.rows), cols = static_cast<uint32_t>(a.cols);
    const uint32_t gpr = cols >> a.w.lg_group;
    // The thread's row of the block of the weight, and which half of the columns: eight lanes in a row
    // write eight different 16-byte pieces of the swizzled lines (no bank conflicts).
    const uint32_t row16 = (lane & 7) + 8 * (lane >> 4), r = 16 * wi + row16, half = (lane >> 3) & 1;
    const uint32_t cc = (MATS == 2 ? 32 : 64) * half;
    uint8_t* ring = smem + a.p.off_ring + (warp - 2) * (kDepth * MATS * kTile);
    const uint32_t ring_u = smem_u32(ring);
    // Where chunk h goes in a stage: line_at + h * line_h, pieces piece0 + h * piece_h ..
    //   linear: the halves are the stage's two tiles, a thread's chunks one line of its tile;
    //   gated: the weights are the two tiles, the halves the two halves of a line;
    //   backward (MN-major): rows 64 .. are the second tile, the halves its two 8 KB blocks of 64
    //   features, a thread's chunks one line.
    const uint32_t line_at = MODE == kMidBackward ? (r >> 6) * kMidTileBytes + half * 8192u + (r & 63) * 128u
                             : MATS == 2          ? r * 128u
                                                  : half * kMidTileBytes + r * 128u;
    const uint32_t line_h = MATS == 2 ? kMidTileBytes : 0u;
    const uint32_t piece0 = MATS == 2 ? 4 * half : 0u;
    constexpr uint32_t piece_h = MATS == 2 ? 0 : 4;

    const uint32_t row_codes = r * cols + cc, row_meta = r * gpr;  // the thread's part of an offset

    // A walk along the group's stages (every second unit of the CTA): where it stands, and how many
    // more of its stages follow in the same tile and weight. Only a new one costs divisions.
    struct Walk {
      uint32_t pos, run, mat, row, col;
    };
    auto enter = [&](Walk& w) {
      const uint32_t tile = (first + w.pos) / KB, kb = first + w.pos - tile * KB;
      const uint32_t block = tile / a.p.tok_tiles * kMidRows;
      uint32_t end = KB;
      w.mat = 0;
      if constexpr (MODE == kMidBackward) {
        const uint32_t kb1 = static_cast<uint32_t>(a.p.kb1);
        w.mat = kb >= kb1 ? 1 : 0;
        if (kb < kb1) end = kb1;
        w.row = (kb - w.mat * kb1) * kBK;
        w.col = block;
      } else {
        w.row = block;
        w.col = kb * kBK;
      }
      w.run = (end - kb + 1) / 2;
    };
    // One stage on; false where that is another tile or weight, and enter() has run.
    auto step = [&](Walk& w) {
      w.pos += 2;
      if constexpr (MODE == kMidBackward)
        w.row += 2 * kBK;
      else
        w.col += 2 * kBK;
      if (--w.run != 0) return true;
      if (w.pos < count) enter(w);
      return false;
    };

    // codes: where the warp's 16 rows begin (3 bits: the 16-byte boundary below) in either weight of a stage
    Walk cw{};
    const uint8_t* copy_base[MATS];
    uint32_t copy_code0[MATS];
    const uint32_t row_step = NBITS == 3 ? cols : cols / 8 * NBITS;
    auto aim_copies = [&]() {
      const int64_t e0 = static_cast<int64_t>(cw.row + 16 * wi) * cols;
#pragma unroll
      for (int i = 0; i < MATS; ++i) {
        copy_base[i] = a.w.packed[MATS == 2 ? i : cw.mat] + (NBITS == 3 ? e0 / 40 * 16 : e0 / 8 * NBITS);
        copy_code0[i] = NBITS == 3 ? static_cast<uint32_t>(e0 % 40) : 0u;
      }
    };
    const int64_t codes_down = static_cast<int64_t>(2 * kBK) * cols / 8 * NBITS;  // two k-blocks of rows
    auto copy_next = [&](uint32_t slot) {
      if (cw.pos < count) {
        if (cw.row + 16 * wi < rows && cw.col < cols) {
          const uint32_t have = min(16u, rows - cw.row - 16 * wi);
          const uint32_t codes = min(static_cast<uint32_t>(kBK), cols - cw.col);
#pragma unroll
          for (int i = 0; i < MATS; ++i)
            Tile::copy(ring_u + (slot * MATS + i) * kTile,
                       copy_base[i] + (NBITS == 3 ? 0u : cw.col / 8 * NBITS), copy_code0[i] + cw.col,
                       row_step, have, codes, lane);
        }
        if (!step(cw) || (MODE == kMidBackward && NBITS == 3))
          aim_copies();
        else if constexpr (MODE == kMidBackward)
          copy_base[0] += codes_down;
      }
      cp_async_commit();
    };
    // scale and zero of the two chunks, a stage ahead
    constexpr int kMeta = kShared ? 1 : 2;
    Walk mw{};
    Slab slab[MATS];
    RawMeta<ANY> next[kMeta][kGroups];
    auto aim = [&]() {
#pragma unroll
      for (int i = 0; i < MATS; ++i)
        slab[i] = slab_of_row<NBITS, ANY>(a.w, MATS == 2 ? i : mw.mat, mw.row, cols, gpr);
    };
    const int64_t meta_down = static_cast<int64_t>(2 * kBK) * gpr * 2;
    auto step_meta = [&]() {
      const bool same = step(mw);
      if (MODE == kMidBackward && same && !ANY && kWhole && NBITS != 3) {
        slab[0].scale += meta_down;
        slab[0].zero += meta_down;
      } else if ((!same || MODE == kMidBackward) && mw.pos < count) {
        aim();
      }
    };
    auto fetch_meta = [&]() {
      if (mw.pos >= count || mw.row + r >= rows) return;
      const uint32_t col = mw.col + cc;
#pragma unroll
      for (int h = 0; h < kMeta; ++h) {
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
          const uint32_t at = col + (MATS == 2 ? 0 : 32 * h) + GROUP * u;
          if (at >= cols) continue;
          const uint32_t group_at = row_meta + (at >> a.w.lg_group);
          if constexpr (!kTwos)
            next[h][u] = load_raw_meta<ANY>(slab[MATS == 2 ? h : 0], a.w, 0u, group_at);
          else if (u % 2 == 0)
            next[h][u] = load_raw_meta_two(slab[MATS == 2 ? h : 0], 0u, group_at);
        }
      }
    };
    mw.pos = cw.pos = group;
    if (group < count) {
      enter(mw);
      aim();
      if constexpr (kWhole) {
        cw = mw;
        aim_copies();
        fetch_meta();
#pragma unroll 1
        for (uint32_t s = 0; s < kDepth; ++s) copy_next(s);
      }
    }
    uint32_t slot = 0, s = group % stages, phase = group >= stages ? 0 : 1;
    while (mw.pos < count) {
      const uint32_t at0 = mw.col + cc, codes0 = row_codes + mw.col;
      const bool in_row = mw.row + r < rows;
      if constexpr (kWhole) {
        GroupMeta m[kMeta][kGroups];
        Exactness known;
#pragma unroll
        for (int h = 0; h < kMeta; ++h)
#pragma unroll
          for (int u = 0; u < kGroups; ++u) {
            RawMeta<ANY> raw = next[h][u];
            if constexpr (kTwos) raw = one_of_two(next[h][u & ~1], u % 2);
            float2 sz = meta_f32_pair<ANY, F16>(raw, slab[MATS == 2 ? h : 0], a.w.meta_dt);
            // W' = 0 outside the weight
            if (!in_row || at0 + (MATS == 2 ? 0 : 32 * h) + GROUP * u >= cols) sz = make_float2(0.0f, 0.0f);
            m[h][u] = group_meta<NBITS, F16>(sz.x, sz.y, &known);
          }
        const bool one = !ANY && __all_sync(0xFFFFFFFFu, known.holds());
        uint32_t first_slot[MATS];  // 3 bits: the row's first code's place in its 16 bytes
#pragma unroll
        for (int i = 0; i < MATS; ++i)
          first_slot[i] = NBITS == 3 ? (slab[i].code0 + codes0 - cc) % 40u : 0u;
        step_meta();
        fetch_meta();
        cp_async_wait<kDepth - 1>();
        __syncwarp();  // every lane's copies have landed
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar(kMidEmpty + s), phase, abort_flag))) break;
        uint8_t* to = smem + s * stage_bytes + line_at;
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
          const int i = MATS == 2 ? h : 0;
          const Codes32<NBITS> c = Tile::read(ring + (slot * MATS + i) * kTile, row16,
                                              cc + (MATS == 2 ? 0 : 32 * h), first_slot[i]);
          uint4 o[4];
          if (one)
            dequant_chunk<NBITS, OUT, kGroups, true>(c, m[kShared ? 0 : h], o);
          else
            dequant_chunk<NBITS, OUT, kGroups, false>(c, m[kShared ? 0 : h], o);
#pragma unroll
          for (uint32_t u = 0; u < 4; ++u)
            *reinterpret_cast<uint4*>(to + h * line_h + (((piece0 + h * piece_h + u) ^ (r & 7)) << 4)) = o[u];
        }
      } else {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar(kMidEmpty + s), phase, abort_flag))) break;
        uint8_t* to = smem + s * stage_bytes + line_at;
#pragma unroll
        for (uint32_t h = 0; h < 2; ++h) {
          const Slab& b = slab[MATS == 2 ? h : 0];
          const uint32_t more = MATS == 2 ? 0 : 32 * h, at = at0 + more;
          const uint32_t left = in_row && at < cols ? min(4u, (cols - at) / 8) : 0u;
          const Codes32<NBITS> c =
              load_codes_units<NBITS>(b.codes, b.code0 + codes0 + more, static_cast<int>(left));
          GroupMeta m[4];
          Exactness known;  // not used
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            float2 sz = make_float2(0.0f, 0.0f);
            if (static_cast<uint32_t>(u) < left)
              sz = meta_f32_pair<ANY, F16>(
                  load_raw_meta<ANY>(b, a.w, 0u, row_meta + ((at + 8 * u) >> a.w.lg_group)), b,
                  a.w.meta_dt);
            m[u] = group_meta<NBITS, F16>(sz.x, sz.y, &known);
          }
          uint4 o[4];
          dequant_chunk<NBITS, OUT, 4, false>(c, m, o);
#pragma unroll
          for (uint32_t u = 0; u < 4; ++u)
            *reinterpret_cast<uint4*>(to + h * line_h + (((piece0 + h * piece_h + u) ^ (r & 7)) << 4)) = o[u];
        }
        step_meta();
      }
      fence_proxy_async_smem();  // generic-proxy writes -> read by the tensor core
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kMidFull + s));
      s += 2;  // the other group fills the stage between
      if (s >= stages) {
        s -= stages;
        phase ^= 1;
      }
      if constexpr (kWhole) {
        copy_next(slot);
        slot = slot + 1 == kDepth ? 0 : slot + 1;
      }
    }
    if constexpr (kWhole) cp_async_wait<0>();
  } else {
    // ------------------------------------------------------------ epilogue
    const uint32_t quarter = warp & 3;  // the TMEM lanes this warp may read
    const uint32_t row = quarter * 32 + lane;
    uint32_t tile = first / KB, kb = first - tile * KB, left = count;
    bool lost = false;  // a wait ran out: this and all later sums
    for (uint32_t seg = 0; left > 0; ++seg) {
      const uint32_t n_kb = min(KB - kb, left), buf = seg % bufs;
      const bool whole = n_kb == KB;
      lost = lost || !__all_sync(0xFFFFFFFFu, mbar_wait_idle(bar(kMidAccFull + buf), (seg / bufs) & 1,
                                                             abort_flag) &&
                                                  !*abort_flag);
      const int n = static_cast<int>(tile / a.p.tok_tiles * kMidRows + row);
      const int64_t tok0 = static_cast<int64_t>(tile % a.p.tok_tiles) * T;
      float* part = a.partial + static_cast<size_t>(2 * blockIdx.x + (seg == 0 ? 0 : 1)) * MATS * T *
                                    kMidRows + row;
      if (lost) {
        if (!whole) {
#pragma unroll 1
          for (uint32_t t = 0; t < T; ++t) part[t * kMidRows] = __uint_as_float(kNoPart);
        }
        left -= n_kb;
        kb = 0;
        ++tile;
        continue;
      }
      tc_fence_after();
      const uint32_t base = tmem + ((quarter * 32) << 16) + buf * MATS * T;
#pragma unroll 1
      for (uint32_t t = 0; t < T; t += 16) {
        uint32_t g[16], u[16];
        mid_tmem_ld16(base + t, g);
        if constexpr (MATS == 2) mid_tmem_ld16(base + T + t, u);
#pragma unroll
        for (uint32_t i = 0; i < 16; ++i) {
          if (!whole) {
            part[(t + i) * kMidRows] = __uint_as_float(g[i]);
            if constexpr (MATS == 2) part[(T + t + i) * kMidRows] = __uint_as_float(u[i]);
          } else if (n < a.out && tok0 + t + i < a.M) {
            mid_store<F16, MATS>(a, tok0 + t + i, n, __uint_as_float(g[i]),
                                 MATS == 2 ? __uint_as_float(u[i]) : 0.0f);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kMidAccEmpty + buf));
      left -= n_kb;
      kb = 0;
      ++tile;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u)
                 : "memory");
  }
}

// Tiles that several CTAs share: their partial tiles added in the order of k, then the epilogue.
// A block takes 8 tokens of a tile, a warp one of them, a lane 4 outputs. Launched while the
// product runs (programmatic dependent launch; 32 registers, so that blocks fit beside it): it finds
// its place first and then waits for the product's end.
template <bool F16, int MATS>
__global__ void __launch_bounds__(256, 8) mid_finish_kernel(const MidArgs a) {
  const uint32_t T = static_cast<uint32_t>(a.p.tok), KB = static_cast<uint32_t>(a.p.kb);
  const uint32_t ctas = static_cast<uint32_t>(a.p.ctas);
  const uint32_t units = static_cast<uint32_t>(a.p.row_tiles * a.p.tok_tiles) * KB;
  const uint32_t tile = blockIdx.x;
  const uint32_t c0 = mid_cta_of(tile * KB, ctas, units);
  const uint32_t c1 = mid_cta_of(tile * KB + KB - 1, ctas, units);
  // c0 may have begun with an earlier tile (then this one is its last); the others begin with this
  const uint32_t slot0 = 2 * c0 + (mid_first_unit(c0, ctas, units) / KB != tile ? 1 : 0);
  const uint32_t row = (threadIdx.x & 31) * 4, t = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int n = static_cast<int>(tile / a.p.tok_tiles * kMidRows + row);
  const int64_t tok = static_cast<int64_t>(tile % a.p.tok_tiles) * T + t;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (c0 == c1 || n >= a.out || t >= T || tok >= a.M) return;
  const size_t slot = static_cast<size_t>(MATS) * T * kMidRows;
  float4 s[MATS];
#pragma unroll
  for (int m = 0; m < MATS; ++m)
    s[m] = __ldcg(reinterpret_cast<const float4*>(
        a.partial + slot0 * slot + (static_cast<size_t>(m) * T + t) * kMidRows + row));
  bool whole = __float_as_uint(s[0].x) != kNoPart;  // (one warp writes, or gives up, all four)
#pragma unroll 2
  for (uint32_t c = c0 + 1; c <= c1; ++c) {
#pragma unroll
    for (int m = 0; m < MATS; ++m) {
      const float4 p = __ldcg(reinterpret_cast<const float4*>(
          a.partial + 2 * c * slot + (static_cast<size_t>(m) * T + t) * kMidRows + row));
      if (m == 0) whole = whole && __float_as_uint(p.x) != kNoPart;
      s[m] = make_float4(__fadd_rn(s[m].x, p.x), __fadd_rn(s[m].y, p.y), __fadd_rn(s[m].z, p.z),
                         __fadd_rn(s[m].w, p.w));
    }
  }
  if (!whole) return;
  const float4 g = s[0], u = s[MATS - 1];
  mid_store<F16, MATS>(a, tok, n, g.x, u.x);
  mid_store<F16, MATS>(a, tok, n + 1, g.y, u.y);
  mid_store<F16, MATS>(a, tok, n + 2, g.z, u.z);
  mid_store<F16, MATS>(a, tok, n + 3, g.w, u.w);
}

// ---------------------------------------------------------------- host side
template <int NBITS, bool F16, int MODE>
cudaError_t launch_mid_mode(const MidJob& j, const MidPlan& plan, cudaStream_t st) {
  const CUtensorMapDataType dt =
      F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int64_t inner = MODE == kMidBackward ? j.rows : j.cols;
  CUtensorMap x[2];
  for (int i = 0; i < 2; ++i) {
    const void* p = MODE == kMidBackward && j.weights == 2 ? j.X[i] : j.X[0];
    if (!make_map(&x[i], dt, 2, p, inner, j.M, 64, static_cast<uint32_t>(plan.tok),
                  CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  MidArgs a = {};
  a.w = weight_args(j.w, j.weights, j.group_size, j.meta_dtype, j.meta_group_size);
  if (MODE == kMidBackward) a.w.bias[0] = a.w.bias[1] = nullptr;
  a.partial = static_cast<float*>(j.workspace);
  a.Y = static_cast<unsigned short*>(j.Y);
  a.G = static_cast<unsigned short*>(j.G);
  a.U = static_cast<unsigned short*>(j.U);
  a.M = static_cast<int>(j.M);
  a.rows = static_cast<int>(j.rows);
  a.cols = static_cast<int>(j.cols);
  a.out = MODE == kMidBackward ? a.cols : a.rows;
  a.act = j.act;
  a.p = plan;
  const bool any = any_meta(j.w, j.weights, j.meta_dtype, j.x_dtype);
  auto kernel = mid_tokens_kernel<NBITS, F16, MODE, 8, true>;
  if (whole_rows(NBITS, j.cols)) {
    if (j.group_size >= 64)
      kernel = any ? mid_tokens_kernel<NBITS, F16, MODE, 64, true>
                   : mid_tokens_kernel<NBITS, F16, MODE, 64, false>;
    else if (j.group_size == 32)
      kernel = any ? mid_tokens_kernel<NBITS, F16, MODE, 32, true>
                   : mid_tokens_kernel<NBITS, F16, MODE, 32, false>;
    else if (j.group_size == 16)  // any, at 2 bits, 8-bit meta, 77 tokens: 36 us against 50 with GROUP 8
      kernel = any || !meta_by_twos(j.w, j.weights) ? mid_tokens_kernel<NBITS, F16, MODE, 16, true>
                                                    : mid_tokens_kernel<NBITS, F16, MODE, 16, false>;
  }
  // always the most, never this call's: a smaller value, set by another thread between here and the
  // launch, would have the launch refused
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMidMaxSmem);
  if (e != cudaSuccess) return e;
  kernel<<<plan.ctas, kMidThreads, plan.smem, st>>>(x[0], x[1], a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (plan.row_tiles * plan.tok_tiles % plan.ctas == 0) return cudaSuccess;  // no tile is shared
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = st;
  cfg.gridDim = dim3(static_cast<unsigned>(plan.row_tiles * plan.tok_tiles),
                     static_cast<unsigned>((plan.tok + 7) / 8));
  cfg.blockDim = dim3(256);
  return cudaLaunchKernelEx(&cfg, mid_finish_kernel<F16, MODE == kMidGated ? 2 : 1>, a);
}

}  // namespace

template <int NBITS>
cudaError_t launch_mid_bits(const MidJob& j, const MidPlan& plan, cudaStream_t st) {
  const bool f16 = j.x_dtype == kF16;
  if (j.mode == kMidLinear)
    return f16 ? launch_mid_mode<NBITS, true, kMidLinear>(j, plan, st)
               : launch_mid_mode<NBITS, false, kMidLinear>(j, plan, st);
  if (j.mode == kMidGated)
    return f16 ? launch_mid_mode<NBITS, true, kMidGated>(j, plan, st)
               : launch_mid_mode<NBITS, false, kMidGated>(j, plan, st);
  return f16 ? launch_mid_mode<NBITS, true, kMidBackward>(j, plan, st)
             : launch_mid_mode<NBITS, false, kMidBackward>(j, plan, st);
}

template <int NBITS>
cudaError_t read_mid_timeouts_bits(unsigned int* out) {
  return cudaMemcpyFromSymbol(out, g_wait_timeouts, sizeof(unsigned int));
}

}  // namespace hqqk
