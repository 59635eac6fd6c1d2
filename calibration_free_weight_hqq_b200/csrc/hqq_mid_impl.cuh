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
//   * Two groups of 8 warps convert codes into the 128-byte-swizzled operand layout, one 128 x 64
//     W' tile (16 KB) after the other: alternate k-blocks, or in the gated form gate and up. A
//     thread converts 32 consecutive codes. Backward the same bytes are an MN-major operand: the
//     contraction runs along the weight's rows, the features along its columns; nothing is
//     transposed.
//   * One warp loads X (TMA, same swizzle), one thread issues the MMAs into TMEM, four warps empty
//     finished accumulators while the next tile runs (two accumulators when TMEM holds them).
//   * Work: all tiles' k-blocks in one line, cut evenly over the CTAs. A CTA that has a tile's whole
//     contraction writes the result; partial tiles go to the workspace in fp32 and a second kernel
//     adds them in order (deterministic).
//   * Codes come by asynchronous copies several tiles ahead, each thread into its own slots; scale and
//     zero one tile ahead in registers.
// Every wait is bounded (about two seconds); on expiry the CTA raises an abort flag, counts the
// timeout, skips its remaining work, waits for its copies in flight and frees its TMEM.
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

constexpr int kMidFullW = 0, kMidEmptyW = kMidFullW + kMidWStages, kMidFullX = kMidEmptyW + kMidWStages,
              kMidEmptyX = kMidFullX + 4, kMidAccFull = kMidEmptyX + 4, kMidAccEmpty = kMidAccFull + 2,
              kMidBars = kMidAccEmpty + 2;

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

// GROUP: 32 (groups of 32 codes or more, cols a multiple of 32), 16 (groups of 16, likewise) or 8 (any
// group size and cols; codes and meta read where they are used). ANY: see RawMeta.
template <int NBITS, bool F16, int MODE, int GROUP, bool ANY>
__global__ void __launch_bounds__(kMidThreads, 1)
    mid_tokens_kernel(const __grid_constant__ CUtensorMap map_x0,
                      const __grid_constant__ CUtensorMap map_x1, const MidArgs a) {
  constexpr int OUT = F16 ? kF16 : kBF16;
  constexpr int MATS = MODE == kMidGated ? 2 : 1;
  constexpr bool kWhole = GROUP != 8;
  constexpr int kGroups = 32 / GROUP;
  constexpr int kDepth = mid_depth(NBITS);
  constexpr int kSlot = 32 * chunk_bytes(NBITS);  // a warp's chunks of a W' tile
  constexpr int kPiece = NBITS == 3 ? 4 : NBITS >= 4 ? 16 : 4 * NBITS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t T = static_cast<uint32_t>(a.p.tok), KB = static_cast<uint32_t>(a.p.kb);
  const uint32_t units = static_cast<uint32_t>(a.p.row_tiles * a.p.tok_tiles) * KB;
  const uint32_t first = mid_first_unit(blockIdx.x, gridDim.x, units);
  const uint32_t count = mid_first_unit(blockIdx.x + 1, gridDim.x, units) - first;
  const uint32_t x_stages = static_cast<uint32_t>(a.p.x_stages), x_bytes = T * (2 * kMidBK);
  const uint32_t bufs = 2 * MATS * T <= 512 ? 2 : 1;
  volatile uint32_t* abort_flag =
      reinterpret_cast<volatile uint32_t*>(smem + a.p.off_bar + 8 * kMidBars + 4);
  auto bar = [&](uint32_t i) { return sbase + a.p.off_bar + 8u * i; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMidWStages; ++s) {
      mbar_init(bar(kMidFullW + s), kMidDqWarps / 2);
      mbar_init(bar(kMidEmptyW + s), 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(bar(kMidFullX + s), 1);
      mbar_init(bar(kMidEmptyX + s), 1);
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
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + a.p.off_bar + 8 * kMidBars);

  if (warp == 0) {
    // ------------------------------------------------------------ X producer
    uint32_t tile = first / KB, kb = first - tile * KB, pos = 0;
    for (; pos < count; ++pos) {
      const uint32_t s = pos % x_stages;
      if (!mbar_wait(bar(kMidEmptyX + s), ((pos / x_stages) & 1) ^ 1, abort_flag)) break;
      if (lane == 0) {
        const bool second = MODE == kMidBackward && kb >= static_cast<uint32_t>(a.p.kb1);
        const int k = static_cast<int>(second ? kb - a.p.kb1 : kb) * kMidBK;
        const int m0 = static_cast<int>((tile % a.p.tok_tiles) * T);
        mbar_arrive_tx(bar(kMidFullX + s), x_bytes);
        tma_load_2d(sbase + a.p.off_x + s * x_bytes, second ? &map_x1 : &map_x0, k, m0,
                    bar(kMidFullX + s));
      }
      __syncwarp();
      if (++kb == KB) {
        kb = 0;
        ++tile;
      }
    }
    if (lane == 0) {  // own copies landed before leaving (complete on the normal path)
      for (uint32_t n = 0; n < x_stages && n < pos; ++n) {
        const uint32_t j = pos - 1 - n;
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(bar(kMidFullX + j % x_stages), (j / x_stages) & 1) &&
               globaltimer() - t0 < kWaitLimitNs) {
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t fmt = F16 ? 0u : 1u;
      constexpr bool kMN = MODE == kMidBackward;
      const uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | (kMN ? 1u << 15 : 0u) |
                             ((T >> 3) << 17) | (static_cast<uint32_t>(kMidRows >> 4) << 24);
      uint32_t kb = first % KB, it = 0, seg = 0;
      bool go = true;
      for (uint32_t pos = 0; pos < count && go; ++pos) {
        const uint32_t buf = seg % bufs;
        const bool begins = pos == 0 || kb == 0;
        if (begins && !mbar_wait(bar(kMidAccEmpty + buf), ((seg / bufs) & 1) ^ 1, abort_flag)) break;
        const uint32_t sx = pos % x_stages;
        if (!mbar_wait(bar(kMidFullX + sx), (pos / x_stages) & 1, abort_flag)) break;
        const uint64_t dx = sw128_kmajor_desc(sbase + a.p.off_x + sx * x_bytes);
#pragma unroll
        for (int m = 0; m < MATS; ++m, ++it) {
          const uint32_t sw = it % kMidWStages;
          if (!mbar_wait(bar(kMidFullW + sw), (it / kMidWStages) & 1, abort_flag)) {
            go = false;
            break;
          }
          tc_fence_after();
          const uint32_t wa = sbase + sw * kMidWBytes;
          const uint64_t dw = kMN ? mid_mnmajor_desc(wa) : sw128_kmajor_desc(wa);
#pragma unroll
          for (int k = 0; k < kMidBK / 16; ++k)
            tc_mma(tmem + (buf * MATS + m) * T, dw + (kMN ? 128 : 2) * k, dx + 2 * k, idesc,
                   !(begins && k == 0));
          tc_commit(bar(kMidEmptyW + sw));
        }
        if (!go) break;
        tc_commit(bar(kMidEmptyX + sx));
        if (++kb == KB || pos + 1 == count) {
          kb = kb == KB ? 0 : kb;
          tc_commit(bar(kMidAccFull + buf));
          ++seg;
        }
      }
      // the issued MMAs have read their operands before the CTA leaves
      for (uint32_t n = 0; n < kMidWStages && n < it; ++n) {
        const uint32_t j = it - 1 - n;
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(bar(kMidEmptyW + j % kMidWStages), (j / kMidWStages) & 1) &&
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
    // the thread's row in the block of weight rows, and its 32 columns in the block of columns
    const uint32_t r = MODE == kMidBackward ? 16 * (wi >> 1) + (lane >> 1) : 16 * wi + (lane >> 1);
    const uint32_t cc = MODE == kMidBackward ? 64 * (wi & 1) + 32 * (lane & 1) : 32 * (lane & 1);
    const uint32_t step = MATS == 2 ? 1 : 2;  // units from one of the group's tiles to its next
    uint8_t* ring = smem + a.p.off_ring + (warp - 2) * (kDepth * kSlot) + lane * kPiece;
    const uint32_t ring_u = smem_u32(ring);
    const uint32_t swz = (MODE == kMidBackward ? (wi & 1) * 8192u : 0u) + r * 128u;

    // Where a walk along the group's tiles stands: unit `pos` of the CTA, its tile and k-block.
    struct Walk {
      uint32_t pos, tile, kb;
    };
    auto start = [&]() {
      Walk w;
      w.pos = MATS == 2 ? 0 : group;
      w.tile = (first + w.pos) / KB;
      w.kb = first + w.pos - w.tile * KB;
      return w;
    };
    auto advance = [&](Walk& w) {
      const uint32_t tile = w.tile;
      w.pos += step;
      w.kb += step;
      while (w.kb >= KB) {
        w.kb -= KB;
        ++w.tile;
      }
      return w.tile != tile;
    };
    // The weight, first row and first column of a unit.
    struct Place {
      uint32_t mat, row, col;
    };
    auto place = [&](const Walk& w) {
      const uint32_t block = w.tile / a.p.tok_tiles * kMidRows;
      Place p;
      if constexpr (MODE == kMidBackward) {
        p.mat = w.kb >= static_cast<uint32_t>(a.p.kb1) ? 1 : 0;
        p.row = (w.kb - p.mat * a.p.kb1) * kMidBK;
        p.col = block;
      } else {
        p.mat = MATS == 2 ? group : 0;
        p.row = block;
        p.col = w.kb * kMidBK;
      }
      return p;
    };

    Walk cw = start(), mw = start(), w = start();
    const uint8_t* copy_base = nullptr;
    uint32_t copy_code0 = 0;
    auto aim_copies = [&]() {
      if (cw.pos < count) {
        const Place p = place(cw);
        const int64_t e0 = static_cast<int64_t>(p.row) * cols;
        copy_base = a.w.packed[p.mat] + (NBITS == 3 ? e0 / 10 * 4 : e0 / 8 * NBITS);
        copy_code0 = NBITS == 3 ? static_cast<uint32_t>(e0 % 10) : 0u;
      }
    };
    auto copy_next = [&](uint32_t slot) {
      if (cw.pos < count) {
        const Place p = place(cw);
        const uint32_t col = p.col + cc;
        if (p.row + r < rows && col < cols) {
          const uint32_t e = r * cols + col;
          if constexpr (NBITS == 3)
            copy_chunk<NBITS>(ring_u + slot * kSlot, copy_base, copy_code0 + e);
          else
            copy_chunk<NBITS>(ring_u + slot * kSlot, copy_base, e / 8 * NBITS);
        }
        if (advance(cw) || MODE == kMidBackward) aim_copies();
      }
      cp_async_commit();
    };
    Slab slab;
    RawMeta<ANY> next[kGroups];
    auto aim = [&]() {
      const Place p = place(mw);
      slab = slab_of_row<NBITS, ANY>(a.w, p.mat, p.row, cols, gpr);
    };
    auto fetch_meta = [&]() {
      if (mw.pos >= count) return;
      const Place p = place(mw);
      const uint32_t col = p.col + cc;
      if (p.row + r >= rows) return;
#pragma unroll
      for (int u = 0; u < kGroups; ++u) {
        if (col + GROUP * u >= cols) break;
        next[u] = load_raw_meta<ANY>(slab, a.w, 0u, r * gpr + ((col + GROUP * u) >> a.w.lg_group));
      }
    };
    if (w.pos < count) {
      aim();
      if constexpr (kWhole) {
        aim_copies();
        fetch_meta();
#pragma unroll 1
        for (uint32_t s = 0; s < kDepth; ++s) copy_next(s);
      }
    }
    uint32_t slot = 0;
    for (; w.pos < count; advance(w)) {
      const uint32_t it = MATS == 2 ? 2 * w.pos + group : w.pos;
      const Place p = place(w);
      const uint32_t col = p.col + cc;
      const bool in = p.row + r < rows && col < cols;
      Codes32<NBITS> c;
      GroupMeta m[kGroups];
      bool one = !ANY;
      if constexpr (kWhole) {
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
          float2 sz = meta_f32_pair<ANY, F16>(next[u], slab, a.w.meta_dt);
          if (!in) sz = make_float2(0.0f, 0.0f);  // W' = 0 outside the weight
          m[u] = group_meta<NBITS>(sz.x, sz.y, &one);
        }
        const uint32_t off = slab.code0 + r * cols + col;
        if (advance(mw) || MODE == kMidBackward) {
          if (mw.pos < count) aim();
        }
        fetch_meta();
        cp_async_wait<kDepth - 1>();  // the thread's own copies: no other reads them
        c = read_chunk<NBITS>(ring + slot * kSlot, off);
      } else {
        const uint32_t left = in ? min(4u, (cols - col) / 8) : 0u;
        if (w.pos != mw.pos) {
          mw = w;
          aim();
        }
        c = load_codes_units<NBITS>(slab.codes, slab.code0 + r * cols + col, static_cast<int>(left));
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
          float2 sz = make_float2(0.0f, 0.0f);
          if (static_cast<uint32_t>(u) < left)
            sz = meta_f32_pair<ANY, F16>(
                load_raw_meta<ANY>(slab, a.w, 0u, r * gpr + ((col + 8 * u) >> a.w.lg_group)), slab,
                a.w.meta_dt);
          m[u] = group_meta<NBITS>(sz.x, sz.y, &one);
        }
      }
      uint4 o[4];
      if (!ANY && __all_sync(0xFFFFFFFFu, one))
        dequant_chunk<NBITS, OUT, kGroups, true>(c, m, o);
      else
        dequant_chunk<NBITS, OUT, kGroups, false>(c, m, o);
      const uint32_t sw = it % kMidWStages;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar(kMidEmptyW + sw), ((it / kMidWStages) & 1) ^ 1,
                                             abort_flag)))
        break;
      uint8_t* tile = smem + sw * kMidWBytes + swz;
#pragma unroll
      for (uint32_t u = 0; u < 4; ++u)
        *reinterpret_cast<uint4*>(tile + (((4 * (lane & 1) + u) ^ (r & 7)) << 4)) = o[u];
      fence_proxy_async_smem();  // generic-proxy writes -> read by the tensor core
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kMidFullW + sw));
      if constexpr (kWhole) {
        copy_next(slot);
        slot = slot + 1 == kDepth ? 0 : slot + 1;
      }
    }
    if constexpr (kWhole) cp_async_wait<0>();
  } else {
    // ------------------------------------------------------------ epilogue
    const uint32_t quarter = warp & 3;  // the TMEM lanes this warp may read
    uint32_t tile = first / KB, kb = first - tile * KB, left = count;
    for (uint32_t seg = 0; left > 0; ++seg) {
      const uint32_t n_kb = min(KB - kb, left), buf = seg % bufs;
      const bool whole = n_kb == KB;
      const bool ok = __all_sync(
          0xFFFFFFFFu, mbar_wait(bar(kMidAccFull + buf), (seg / bufs) & 1, abort_flag) && !*abort_flag);
      if (!ok) break;
      tc_fence_after();
      const uint32_t row = quarter * 32 + lane;
      const int n = static_cast<int>(tile / a.p.tok_tiles * kMidRows + row);
      const int64_t tok0 = static_cast<int64_t>(tile % a.p.tok_tiles) * T;
      float* part = a.partial + static_cast<size_t>(2 * blockIdx.x + (seg == 0 ? 0 : 1)) * MATS * T *
                                    kMidRows + row;
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
// A block takes 8 tokens of a tile.
template <bool F16, int MATS>
__global__ void __launch_bounds__(256) mid_finish_kernel(const MidArgs a) {
  const uint32_t T = static_cast<uint32_t>(a.p.tok), KB = static_cast<uint32_t>(a.p.kb);
  const uint32_t ctas = static_cast<uint32_t>(a.p.ctas);
  const uint32_t units = static_cast<uint32_t>(a.p.row_tiles * a.p.tok_tiles) * KB;
  const uint32_t tile = blockIdx.x;
  const uint32_t c0 = mid_cta_of(tile * KB, ctas, units);
  const uint32_t c1 = mid_cta_of(tile * KB + KB - 1, ctas, units);
  if (c0 == c1) return;  // one CTA had it whole
  const uint32_t row = threadIdx.x & 127;
  const int n = static_cast<int>(tile / a.p.tok_tiles * kMidRows + row);
  if (n >= a.out) return;
  const int64_t tok0 = static_cast<int64_t>(tile % a.p.tok_tiles) * T;
  for (uint32_t i = threadIdx.x >> 7; i < 8; i += 2) {
    const uint32_t t = blockIdx.y * 8 + i;
    if (t >= T || tok0 + t >= a.M) return;
    float s[2] = {0.0f, 0.0f};
    for (uint32_t c = c0; c <= c1; ++c) {
      const uint32_t second = mid_first_unit(c, ctas, units) / KB != tile ? 1 : 0;
      const float* part = a.partial + static_cast<size_t>(2 * c + second) * MATS * T * kMidRows + row;
#pragma unroll
      for (int m = 0; m < MATS; ++m) s[m] = __fadd_rn(s[m], part[(m * T + t) * kMidRows]);
    }
    mid_store<F16, MATS>(a, tok0 + t, n, s[0], s[1]);
  }
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
    if (!make_map(&x[i], dt, 2, p, inner, j.M, kMidBK, static_cast<uint32_t>(plan.tok),
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
  const bool any = any_meta(j.w, j.weights, j.meta_dtype, j.x_dtype), whole = j.cols % 32 == 0;
  auto kernel = mid_tokens_kernel<NBITS, F16, MODE, 8, true>;
  if (j.group_size >= 32)
    kernel = any ? mid_tokens_kernel<NBITS, F16, MODE, 32, true>
                 : mid_tokens_kernel<NBITS, F16, MODE, 32, false>;
  else if (whole && j.group_size == 16 && !any)
    kernel = mid_tokens_kernel<NBITS, F16, MODE, 16, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(plan.smem));
  if (e != cudaSuccess) return e;
  kernel<<<plan.ctas, kMidThreads, plan.smem, st>>>(x[0], x[1], a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (plan.row_tiles * plan.tok_tiles % plan.ctas == 0) return cudaSuccess;  // no tile is shared
  const dim3 grid(static_cast<unsigned>(plan.row_tiles * plan.tok_tiles),
                  static_cast<unsigned>((plan.tok + 7) / 8));
  mid_finish_kernel<F16, MODE == kMidGated ? 2 : 1><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
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
