// hqq_dense.cu - the products of many tokens: tcgen05 matrix products on dequantized weights.
//
// With hundreds of tokens or more the arithmetic outweighs the weight, and a weight dequantized
// once (2 bytes an element, mostly still in L2 when it is read) costs less than converting every
// tile again for each block of tokens. The weight comes from the dequantizer, so W' has its exact
// bits in every format; this kernel multiplies:
//   * forward:   D[M, N] = A[M, K] B[N, K]^T (+ bias)
//   * gated:     D = act(A Bg^T + bg) * (A Bu^T + bu), both products of a tile in one pass over A
//                and the activation and product in its epilogue
//   * backward:  D[M, N] = sum over sources i of A_i[M, K] B_i[K, N]; B is the weight as it lies in
//                memory, rows along the contraction, read by the tensor core as an MN-major operand
//                (no transposed copy); two sources extend the contraction of one accumulator
//
// A CTA pair (cluster of 2, tcgen05 cta_group::2) owns a 256 x 256 accumulator tile at a time:
// each CTA holds 128 rows of A and 128 of the tile's columns of B per k-block of 64, a ring of 6
// stages filled by TMA; the leader's single thread issues the MMAs (M = 256, N = 256, K = 16). Two
// accumulators of 256 TMEM columns alternate, so the epilogue of a tile (four warps: TMEM to
// registers, bias / activation, rounding, TMA stores) runs under the next tile's MMAs. Clusters
// are persistent and visit tiles with the row blocks fastest (16 at a time), so that the
// A panel stays in L2 while each B panel is read once. In the gated form the tile's columns are
// 128 of the gate (the leader's B) and the same 128 of the up projection (the follower's B).
// Where tiles are few the contraction is cut into parts, whose sums a second kernel adds in order.
// What bounds it: the tensor cores, and in long runs the power limit. Measured, 4096 tokens: gated 11008
// x 4096 480-500 us (1480-1540 TFLOP/s, 0.91-0.94 of the library product's burst), gradient of 4096 x
// 11008 235-240 us (1540-1570 TFLOP/s); in a long row of calls, less the other kernels, 588-593 and 288 us
// (1250-1285 TFLOP/s, 0.91-0.93 of the rate that the library product holds for seconds).
//
// Every wait is bounded (about two seconds); on expiry the CTA raises an abort flag, counts the
// timeout, skips its remaining work, waits (bounded) for its copies in flight and frees its TMEM. Its sums of
// parts are marked as missing, and outputs that need one are not written.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <mutex>

#include "hqq_act.cuh"
#include "hqq_device.cuh"
#include "hqq_kernels.h"
#include "hqq_tensor.cuh"
#include "hqq_tiles.h"

namespace hqqk {
namespace {

namespace dense {
constexpr int kBM = 256, kBN = 256, kBK = 64;  // accumulator tile of a pair; k-block
constexpr int kStages = 6;
constexpr int kEpiWarps = 4;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr uint32_t kABytes = 128 * kBK * 2;    // one CTA's half of A
constexpr uint32_t kBBytes = 128 * kBK * 2;    // one CTA's half of B
constexpr uint32_t kBHalf = 64 * kBK * 2;      // MN-major: 64 columns x 64 contraction rows
constexpr uint32_t kOffA = 0;
constexpr uint32_t kOffB = kOffA + kStages * kABytes;
constexpr uint32_t kBlockBytes = 32 * 32 * 2;  // an output block of the epilogue
constexpr int kBlocks = 3;                     // staged blocks per epilogue warp
constexpr uint32_t kOffOut = kOffB + kStages * kBBytes;
constexpr uint32_t kOffBar = kOffOut + kEpiWarps * kBlocks * kBlockBytes;
constexpr int kFull = 0, kEmpty = kStages, kAccFull = 2 * kStages, kAccEmpty = kAccFull + 2;
constexpr int kNumBars = kAccEmpty + 2;
constexpr uint32_t kOffTmem = kOffBar + 8 * kNumBars;
constexpr uint32_t kOffAbort = kOffTmem + 4;
constexpr uint32_t kSmemBytes = kOffAbort + 4 + 1024;
constexpr uint32_t kTmemCols = 512;
constexpr int kGroupM = 16;  // row blocks visited before the next column block
static_assert(kOffB % 1024 == 0 && kBBytes % 1024 == 0, "SW128 tiles");
static_assert(kOffOut % 1024 == 0, "SW64 blocks");
static_assert(kSmemBytes <= 232448, "shared memory per CTA");
}  // namespace dense

struct DenseArgs {
  const unsigned short* bias[2];
  int M, N, K;          // output rows and columns, contraction of one source
  int sources;
  int tiles_m, tiles_n;
  int splits, kb_split;  // parts of the contraction, k-blocks of a part
  float* partial;        // of more than one part: [part][products][M][N]
  unsigned short *D, *G, *U;
  int act;
  bool save_g, save_u;
};

// Shared-memory descriptor of an MN-major operand tile in the 128-byte swizzle: lines of 64
// elements along MN (128 B), one line per contraction index, 8-line atoms 1024 B apart along the
// contraction (stride byte offset) and blocks of 64 MN elements kBHalf apart (leading byte
// offset). Other fields as in sw128_kmajor_desc.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) |
         (static_cast<uint64_t>(dense::kBHalf >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// kind::f16, fp32 accumulator, M = 256, N = 256; bit 16: B is MN-major.
template <bool F16, bool BMN>
__device__ __forceinline__ uint32_t dense_idesc() {
  constexpr uint32_t fmt = F16 ? 0u : 1u;
  return (1u << 4) | (fmt << 7) | (fmt << 10) | (BMN ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(dense::kBN >> 3) << 17) |
         (static_cast<uint32_t>(dense::kBM >> 4) << 24);
}

// Tile index -> (row block, column block): row blocks fastest inside bands of kGroupM. The parts of
// the contraction follow one another.
__device__ __forceinline__ void tile_coords(int tile, const DenseArgs& a, int* tm, int* tn) {
  tile %= a.tiles_m * a.tiles_n;
  const int band = tile / (dense::kGroupM * a.tiles_n);
  const int first = band * dense::kGroupM;
  const int rows = min(dense::kGroupM, a.tiles_m - first);
  const int in = tile - band * dense::kGroupM * a.tiles_n;
  *tn = in / rows;
  *tm = first + in - *tn * rows;
}

// One 32 x 32 output block of a warp: rounded, staged with the 64-byte swizzle, stored by TMA
// (rows past M and columns past N are clipped by the copy).
template <int OUT>
__device__ __forceinline__ void store_block(const CUtensorMap* map, uint8_t* stage, int lane,
                                            const uint32_t (&o)[16], int x, int y) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *reinterpret_cast<uint4*>(stage + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) =
        make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(map, smem_u32(stage), x, y);
    bulk_commit();
  }
}

// Where the part of a tile's row `row` from column n0 on would go: marked as missing, every four columns.
template <int PRODUCTS>
__device__ __forceinline__ void no_part(const DenseArgs& a, int part, int64_t row, int n0, int columns) {
  if (row >= a.M) return;
  float* to = a.partial + (static_cast<int64_t>(part) * PRODUCTS * a.M + row) * a.N;
#pragma unroll 1
  for (int n = n0; n < n0 + columns && n < a.N; n += 4) to[n] = __uint_as_float(kNoPart);
}

template <bool F16>
__device__ __forceinline__ float bias_at(const unsigned short* bias, int n, int N) {
  if (bias == nullptr || n >= N) return 0.0f;
  return F16 ? f16_bits_to_f32(__ldg(bias + n)) : bf16_bits_to_f32(__ldg(bias + n));
}

template <bool F16, int KIND, int ACT>
__global__ void __launch_bounds__(dense::kThreads, 1)
    dense_2sm_kernel(const __grid_constant__ CUtensorMap map_a0,
                     const __grid_constant__ CUtensorMap map_a1,
                     const __grid_constant__ CUtensorMap map_b0,
                     const __grid_constant__ CUtensorMap map_b1,
                     const __grid_constant__ CUtensorMap map_d,
                     const __grid_constant__ CUtensorMap map_g,
                     const __grid_constant__ CUtensorMap map_u, const DenseArgs args) {
  using namespace dense;
  constexpr int OUT = F16 ? kF16 : kBF16;
  constexpr bool kMN = KIND == kDenseBackward;
  constexpr int kTileN = KIND == kDenseGated ? kBN / 2 : kBN;  // output columns per tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();  // 0: leader, issues the MMAs
  const bool leader = rank == 0;
  const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
  const int tiles = args.tiles_m * args.tiles_n * args.splits;
  const int KB1 = (args.K + kBK - 1) / kBK;
  const int KB = KB1 * args.sources;
  // the k-blocks of a tile's part
  auto part_begin = [&](int tile) { return tile / (args.tiles_m * args.tiles_n) * args.kb_split; };
  auto part_end = [&](int tile) { return min(KB, part_begin(tile) + args.kb_split); };
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + kOffAbort);
  auto bar = [&](int i) { return sbase + kOffBar + 8u * static_cast<uint32_t>(i); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(kFull + s), 1);   // leader: expect_tx for both CTAs' copies
      mbar_init(bar(kEmpty + s), 1);  // leader's commit, in both CTAs
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kAccFull + i), 1);               // leader's commit, in both CTAs
      mbar_init(bar(kAccEmpty + i), 2 * kEpiWarps);  // leader: the epilogue warps of both CTAs
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {  // the same warp in both CTAs, as the paired allocation requires
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     sbase + kOffTmem),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // barriers of both CTAs initialised, TMEM address written in both
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + kOffTmem);
  const uint32_t leader_bars = cluster_addr(sbase + kOffBar, 0);
  auto lbar = [&](int i) { return leader_bars + 8u * static_cast<uint32_t>(i); };

  // dense_finish_kernel may take its place now; it waits for this grid's end before it reads
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == 0) {
    // ------------------------------------------------------------ producer (both CTAs)
    int it = 0;
    bool go = true;
    for (int tile = pair; tile < tiles && go; tile += pairs) {
      int tm, tn;
      tile_coords(tile, args, &tm, &tn);
      const int m0 = tm * kBM + static_cast<int>(rank) * 128;
      const int n0 = tn * kTileN + (KIND == kDenseGated ? 0 : static_cast<int>(rank) * 128);
      const int end = part_end(tile);
      for (int kb = part_begin(tile); kb < end; ++kb, ++it) {
        const int s = it % kStages;
        if (!mbar_wait_cl(bar(kEmpty + s), ((it / kStages) & 1) ^ 1, abort_flag)) {
          go = false;
          break;
        }
        if (lane == 0) {
          if (leader) mbar_arrive_tx(bar(kFull + s), 2 * (kABytes + kBBytes));
          const uint32_t a = sbase + kOffA + s * kABytes, b = sbase + kOffB + s * kBBytes;
          const uint32_t full = lbar(kFull + s);
          const bool second = KIND == kDenseBackward && kb >= KB1;
          const int k = (second ? kb - KB1 : kb) * kBK;
          tma_load_2d_pair(a, second ? &map_a1 : &map_a0, k, m0, full);
          if constexpr (kMN) {
            const CUtensorMap* mb = second ? &map_b1 : &map_b0;
            tma_load_2d_pair(b, mb, n0, k, full);
            tma_load_2d_pair(b + kBHalf, mb, n0 + 64, k, full);
          } else {
            tma_load_2d_pair(b, KIND == kDenseGated && !leader ? &map_b1 : &map_b0, k, n0, full);
          }
        }
        __syncwarp();
      }
    }
    if (leader && lane == 0) {  // both CTAs' copies landed before the pair parts
      for (int j = it - 1; j >= 0 && j >= it - kStages; --j) {
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait_cluster(bar(kFull + j % kStages), (j / kStages) & 1) &&
               globaltimer() - t0 < kWaitLimitNs) {
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int it = 0;
      if (leader) {
        // -------------------------------------------------------- MMA issuer
        const uint32_t idesc = dense_idesc<F16, kMN>();
        int n = 0;
        bool go = true;
        for (int tile = pair; tile < tiles && go; tile += pairs, ++n) {
          const uint32_t acc = n & 1;
          if (!mbar_wait_cl(bar(kAccEmpty + acc), ((n >> 1) & 1) ^ 1, abort_flag)) break;
          tc_fence_after();
          const int begin = part_begin(tile), end = part_end(tile);
          for (int kb = begin; kb < end; ++kb, ++it) {
            const int s = it % kStages;
            if (!mbar_wait_cl(bar(kFull + s), (it / kStages) & 1, abort_flag)) {
              go = false;
              break;
            }
            tc_fence_after();
            const uint64_t da = sw128_kmajor_desc(sbase + kOffA + s * kABytes);
            const uint32_t b = sbase + kOffB + s * kBBytes;
            const uint64_t db = kMN ? sw128_mnmajor_desc(b) : sw128_kmajor_desc(b);
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k)
              tc_mma_pair(tmem + acc * kBN, da + 2 * k, db + (kMN ? 128 : 2) * k, idesc,
                          kb != begin || k != 0);
            tc_commit_pair(bar(kEmpty + s));
          }
          if (go) tc_commit_pair(bar(kAccFull + acc));
        }
      } else {
        for (int tile = pair; tile < tiles; tile += pairs) it += part_end(tile) - part_begin(tile);
      }
      // The commits land in both CTAs' barriers asynchronously: see the last use of every stage
      // completed before the pair parts (a bounded wait; after an abort it may run out).
      for (int j = it - 1; j >= 0 && j >= it - kStages; --j) {
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait_cluster(bar(kEmpty + j % kStages), (j / kStages) & 1) &&
               (leader || !*abort_flag) && globaltimer() - t0 < 2 * kWaitLimitNs) {
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int quarter = warp & 3;  // the TMEM lanes this warp may read
    uint8_t* stage = smem + kOffOut + static_cast<uint32_t>(warp - 2) * kBlocks * kBlockBytes;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    int n = 0;
    uint32_t stored = 0;  // blocks of this warp, over all its tiles
    bool lost = false;    // a wait ran out: this and all later tiles
    for (int tile = pair; tile < tiles; tile += pairs, ++n) {
      const uint32_t acc = n & 1;
      lost = lost || !__all_sync(0xFFFFFFFFu, mbar_wait_cl(bar(kAccFull + acc), (n >> 1) & 1,
                                                           abort_flag) &&
                                                  !*abort_flag);
      int tm, tn;
      tile_coords(tile, args, &tm, &tn);
      const int row0 = tm * kBM + static_cast<int>(rank) * 128 + quarter * 32;
      if (lost) {
        if (args.splits == 1) break;
        no_part<KIND == kDenseGated ? 2 : 1>(args, tile / (args.tiles_m * args.tiles_n), row0 + lane,
                                             tn * kTileN, kTileN);
        continue;
      }
      tc_fence_after();
      const uint32_t base = tmem + lanes + acc * kBN;
#pragma unroll 1
      for (int c = 0; c < kTileN / 32; ++c) {
        const int nc = tn * kTileN + c * 32;
        const bool in = nc < args.N && row0 < args.M;
        uint32_t r[32], o[16];
        tmem_ld32(base + c * 32, r);
        if (args.splits > 1) {  // a part: 32 columns of this lane's row, unrounded
          constexpr int kProducts = KIND == kDenseGated ? 2 : 1;
          const int64_t part = tile / (args.tiles_m * args.tiles_n), row = row0 + lane;
#pragma unroll
          for (int m = 0; m < kProducts; ++m) {
            if (m == 1) tmem_ld32(base + kTileN + c * 32, r);
            float* to = args.partial + ((part * kProducts + m) * args.M + row) * args.N + nc;
#pragma unroll
            for (int i = 0; i < 32; i += 4)  // N is a multiple of 8
              if (row < args.M && nc + i < args.N)
                *reinterpret_cast<uint4*>(to + i) = make_uint4(r[i], r[i + 1], r[i + 2], r[i + 3]);
          }
          continue;
        }
        if constexpr (KIND == kDenseGated) {
          uint32_t r2[32], og[16], ou[16];
          tmem_ld32(base + kTileN + c * 32, r2);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float g0 = __fadd_rn(__uint_as_float(r[i]), bias_at<F16>(args.bias[0], nc + i, args.N));
            const float g1 = __fadd_rn(__uint_as_float(r[i + 1]), bias_at<F16>(args.bias[0], nc + i + 1, args.N));
            const float u0 = __fadd_rn(__uint_as_float(r2[i]), bias_at<F16>(args.bias[1], nc + i, args.N));
            const float u1 = __fadd_rn(__uint_as_float(r2[i + 1]), bias_at<F16>(args.bias[1], nc + i + 1, args.N));
            og[i / 2] = pack2_16<OUT>(g0, g1);
            ou[i / 2] = pack2_16<OUT>(u0, u1);
            o[i / 2] = pack2_16<OUT>(__fmul_rn(act_f32<ACT>(g0), u0), __fmul_rn(act_f32<ACT>(g1), u1));
          }
          if (lane == 0) bulk_wait_read<0>();  // the previous blocks have left their staging
          __syncwarp();
          if (in) {
            store_block<OUT>(&map_d, stage, lane, o, nc, row0);
            if (args.save_g) store_block<OUT>(&map_g, stage + kBlockBytes, lane, og, nc, row0);
            if (args.save_u) store_block<OUT>(&map_u, stage + 2 * kBlockBytes, lane, ou, nc, row0);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float v0 = __uint_as_float(r[i]), v1 = __uint_as_float(r[i + 1]);
            if (KIND == kDenseForward) {
              v0 = __fadd_rn(v0, bias_at<F16>(args.bias[0], nc + i, args.N));
              v1 = __fadd_rn(v1, bias_at<F16>(args.bias[0], nc + i + 1, args.N));
            }
            o[i / 2] = pack2_16<OUT>(v0, v1);
          }
          // The last store may still be read, so the slots alternate by stored blocks: by c, the first block
          // of a tile would take the slot of a tile's last one that N cut off at an even c.
          if (lane == 0) bulk_wait_read<1>();
          __syncwarp();
          if (in) store_block<OUT>(&map_d, stage + (stored++ & 1) * kBlockBytes, lane, o, nc, row0);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(lbar(kAccEmpty + acc));
    }
    if (lane == 0) bulk_wait_read<0>();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  }
}

// The parts of a product added in order, then its epilogue; four outputs a thread. Launched while the
// product runs (programmatic dependent launch); waits for its end first.
template <bool F16, int KIND>
__global__ void __launch_bounds__(256, 4) dense_finish_kernel(const DenseArgs a) {
  constexpr int OUT = F16 ? kF16 : kBF16;
  constexpr int kProducts = KIND == kDenseGated ? 2 : 1;
  const int64_t plane = static_cast<int64_t>(a.M) * a.N;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int64_t at = (blockIdx.x * static_cast<int64_t>(256) + threadIdx.x) * 4; at < plane;
       at += static_cast<int64_t>(gridDim.x) * 1024) {
    float s[kProducts][4] = {};
    bool whole = true;
    for (int p = 0; p < a.splits; ++p) {
#pragma unroll
      for (int m = 0; m < kProducts; ++m) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(a.partial + (p * kProducts + m) * plane + at));
        if (m == 0) whole = whole && __float_as_uint(v.x) != kNoPart;
        s[m][0] = __fadd_rn(s[m][0], v.x);
        s[m][1] = __fadd_rn(s[m][1], v.y);
        s[m][2] = __fadd_rn(s[m][2], v.z);
        s[m][3] = __fadd_rn(s[m][3], v.w);
      }
    }
    if (!whole) continue;
    const int n = static_cast<int>(at % a.N);
    float y[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      y[q] = s[0][q];
      if constexpr (KIND != kDenseBackward) y[q] = __fadd_rn(y[q], bias_at<F16>(a.bias[0], n + q, a.N));
      if constexpr (KIND == kDenseGated) {
        s[0][q] = y[q];
        s[1][q] = __fadd_rn(s[1][q], bias_at<F16>(a.bias[1], n + q, a.N));
        const float h = a.act == kSilu   ? act_f32<kSilu>(y[q])
                        : a.act == kGelu ? act_f32<kGelu>(y[q])
                                         : act_f32<kGeluTanh>(y[q]);
        y[q] = __fmul_rn(h, s[1][q]);
      }
    }
    auto four = [&](unsigned short* to, const float* v) {
      *reinterpret_cast<uint2*>(to + at) = make_uint2(pack2_16<OUT>(v[0], v[1]), pack2_16<OUT>(v[2], v[3]));
    };
    four(a.D, y);
    if constexpr (KIND == kDenseGated) {
      if (a.G != nullptr) four(a.G, s[0]);
      if (a.U != nullptr) four(a.U, s[1]);
    }
  }
}

// ---------------------------------------------------------------- host side
// Resident pairs of `kernel` on the current device (cached per kernel and device).
int resident_pairs(const void* kernel) {
  struct Entry { const void* k; int dev, n; };
  static std::mutex mu;
  static Entry cache[128];
  static int used = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < used; ++i)
    if (cache[i].k == kernel && cache[i].dev == dev) return cache[i].n;
  cudaLaunchConfig_t c = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = 1;
  c.gridDim = dim3(2);
  c.blockDim = dim3(dense::kThreads);
  c.dynamicSmemBytes = dense::kSmemBytes;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &c) != cudaSuccess || n < 1) {
    (void)cudaGetLastError();
    n = 64;  // more clusters than fit only means that some wait for their turn
  }
  if (used < 128) cache[used++] = Entry{kernel, dev, n};
  return n;
}

template <bool F16, int KIND, int ACT>
cudaError_t launch_dense_typed(const DenseJob& j, cudaStream_t st) {
  const CUtensorMapDataType dt =
      F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  auto kernel = dense_2sm_kernel<F16, KIND, ACT>;
  CUtensorMap a[2], b[2], d, g, u;
  const auto sw128 = CU_TENSOR_MAP_SWIZZLE_128B, sw64 = CU_TENSOR_MAP_SWIZZLE_64B;
  const int na = KIND == kDenseBackward ? j.sources : 1;
  const int nb = KIND == kDenseForward ? 1 : KIND == kDenseGated ? 2 : j.sources;
  bool ok = true;
  for (int i = 0; i < 2; ++i) {
    const int ia = i < na ? i : 0, ib = i < nb ? i : 0;
    ok = ok && make_map(&a[i], dt, 2, j.A[ia], j.K, j.M, dense::kBK, 128, sw128);
    ok = ok && (KIND == kDenseBackward
                    ? make_map(&b[i], dt, 2, j.B[ib], j.N, j.K, 64, dense::kBK, sw128)
                    : make_map(&b[i], dt, 2, j.B[ib], j.K, j.N, dense::kBK, 128, sw128));
  }
  ok = ok && make_map(&d, dt, 2, j.D, j.N, j.M, 32, 32, sw64);
  ok = ok && make_map(&g, dt, 2, j.G != nullptr ? j.G : j.D, j.N, j.M, 32, 32, sw64);
  ok = ok && make_map(&u, dt, 2, j.U != nullptr ? j.U : j.D, j.N, j.M, 32, 32, sw64);
  if (!ok) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(dense::kSmemBytes));
  if (e != cudaSuccess) return e;
  DenseArgs args = {};
  args.bias[0] = static_cast<const unsigned short*>(j.bias[0]);
  args.bias[1] = static_cast<const unsigned short*>(j.bias[1]);
  args.M = static_cast<int>(j.M);
  args.N = static_cast<int>(j.N);
  args.K = static_cast<int>(j.K);
  args.sources = KIND == kDenseBackward ? j.sources : 1;
  const int tile_n = KIND == kDenseGated ? dense::kBN / 2 : dense::kBN;
  const int64_t tm = (j.M + dense::kBM - 1) / dense::kBM, tn = (j.N + tile_n - 1) / tile_n;
  if (tm * tn > 0x3FFFFFFF) return cudaErrorInvalidValue;
  args.tiles_m = static_cast<int>(tm);
  args.tiles_n = static_cast<int>(tn);
  const int KB = static_cast<int>((j.K + dense::kBK - 1) / dense::kBK) * args.sources;
  args.splits = dense_splits(j.kind, j.M, j.N, j.K, j.sources);
  args.kb_split = (KB + args.splits - 1) / args.splits;
  args.splits = (KB + args.kb_split - 1) / args.kb_split;  // no empty part
  args.partial = static_cast<float*>(j.partial);
  args.D = static_cast<unsigned short*>(j.D);
  args.G = static_cast<unsigned short*>(j.G);
  args.U = static_cast<unsigned short*>(j.U);
  args.act = j.act;
  args.save_g = j.G != nullptr;
  args.save_u = j.U != nullptr;
  const int64_t pairs =
      std::min<int64_t>(tm * tn * args.splits, resident_pairs(reinterpret_cast<const void*>(kernel)));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = st;
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(dense::kThreads);
  cfg.dynamicSmemBytes = dense::kSmemBytes;
  e = cudaLaunchKernelEx(&cfg, kernel, a[0], a[1], b[0], b[1], d, g, u, args);
  if (e != cudaSuccess || args.splits == 1) return e;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>((j.M * j.N / 4 + 255) / 256, kSms * 8)));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, dense_finish_kernel<F16, KIND>, args);
}

template <bool F16>
cudaError_t launch_dense_kind(const DenseJob& j, cudaStream_t st) {
  if (j.kind == kDenseForward) return launch_dense_typed<F16, kDenseForward, kSilu>(j, st);
  if (j.kind == kDenseBackward) return launch_dense_typed<F16, kDenseBackward, kSilu>(j, st);
  if (j.act == kSilu) return launch_dense_typed<F16, kDenseGated, kSilu>(j, st);
  if (j.act == kGelu) return launch_dense_typed<F16, kDenseGated, kGelu>(j, st);
  return launch_dense_typed<F16, kDenseGated, kGeluTanh>(j, st);
}

// ---------------------------------------------------------------- elementwise gradient
// dG = dY U act'(G), dU = dY act(G): 10 bytes moved per element, HBM bound. 8 elements a thread.
template <bool F16, int ACT>
__global__ void __launch_bounds__(256)
    gated_grad_kernel(const uint4* dY, const uint4* G, const uint4* U, uint4* dG, uint4* dU,
                      int64_t n8) {
  constexpr int OUT = F16 ? kF16 : kBF16;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(256) + threadIdx.x; i < n8;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const uint4 vy = __ldg(dY + i), vg = __ldg(G + i), vu = __ldg(U + i);
    const uint32_t y[4] = {vy.x, vy.y, vy.z, vy.w}, g[4] = {vg.x, vg.y, vg.z, vg.w},
                   u[4] = {vu.x, vu.y, vu.z, vu.w};
    uint32_t og[4], ou[4];
    auto half = [](uint32_t w, int h) {
      const uint32_t b = h ? w >> 16 : w & 0xFFFFu;
      return F16 ? f16_bits_to_f32(b) : bf16_bits_to_f32(b);
    };
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float dg[2], du[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float d = half(y[q], h);
        const float2 a = act_and_grad_f32<ACT>(half(g[q], h));
        dg[h] = d * half(u[q], h) * a.y;
        du[h] = d * a.x;
      }
      og[q] = pack2_16<OUT>(dg[0], dg[1]);
      ou[q] = pack2_16<OUT>(du[0], du[1]);
    }
    dG[i] = make_uint4(og[0], og[1], og[2], og[3]);
    dU[i] = make_uint4(ou[0], ou[1], ou[2], ou[3]);
  }
}

template <bool F16>
cudaError_t launch_gated_grad_typed(const void* dY, const void* G, const void* U, int64_t n,
                                    int act, void* dG, void* dU, cudaStream_t st) {
  const int64_t n8 = n / 8;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>((n8 + 255) / 256, 148 * 8));
  const uint4 *y = static_cast<const uint4*>(dY), *g = static_cast<const uint4*>(G),
              *u = static_cast<const uint4*>(U);
  uint4 *og = static_cast<uint4*>(dG), *ou = static_cast<uint4*>(dU);
  if (act == kSilu)
    gated_grad_kernel<F16, kSilu><<<grid, 256, 0, st>>>(y, g, u, og, ou, n8);
  else if (act == kGelu)
    gated_grad_kernel<F16, kGelu><<<grid, 256, 0, st>>>(y, g, u, og, ou, n8);
  else
    gated_grad_kernel<F16, kGeluTanh><<<grid, 256, 0, st>>>(y, g, u, og, ou, n8);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- empty sums
template <bool F16>
__global__ void __launch_bounds__(256)
    empty_sums_kernel(const unsigned short* bg, const unsigned short* bu, int mats, int64_t total,
                      int64_t N, int act, unsigned short* Y, unsigned short* G, unsigned short* U) {
  constexpr int OUT = F16 ? kF16 : kBF16;
  auto bits = [](float f) { return static_cast<unsigned short>(pack2_16<OUT>(f, 0.0f)); };
  for (int64_t i = blockIdx.x * static_cast<int64_t>(256) + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t n = i % N;
    const unsigned short hg = bg != nullptr ? bg[n] : 0, hu = bu != nullptr ? bu[n] : 0;
    if (mats == 1) {
      Y[i] = hg;
      continue;
    }
    const float g = F16 ? f16_bits_to_f32(hg) : bf16_bits_to_f32(hg);
    const float u = F16 ? f16_bits_to_f32(hu) : bf16_bits_to_f32(hu);
    const float h = act == kSilu   ? act_f32<kSilu>(g)
                    : act == kGelu ? act_f32<kGelu>(g)
                                   : act_f32<kGeluTanh>(g);
    Y[i] = bits(__fmul_rn(h, u));
    if (G != nullptr) G[i] = hg;
    if (U != nullptr) U[i] = hu;
  }
}

// ---------------------------------------------------------------- column sums
// Up to two matrices of one shape (blockIdx.y). A block owns 32 columns: 4 threads of 8 columns side by
// side (64 bytes), 64 rows at a time; each thread adds its rows in order, eight loads in flight, then
// the 64 partial sums are added in order. Bound: the latency of those loads (4096 x 4096: 10.6 us, 3.2
// TB/s; both of a pair, 129 x 11008, in one launch: 4.5 us).
template <bool F16>
__global__ void __launch_bounds__(256)
    column_sums_kernel(const unsigned short* A0, unsigned short* out0, const unsigned short* A1,
                       unsigned short* out1, int64_t rows, int64_t cols) {
  constexpr int OUT = F16 ? kF16 : kBF16;
  const unsigned short* A = blockIdx.y == 0 ? A0 : A1;
  unsigned short* out = blockIdx.y == 0 ? out0 : out1;
  if (out == nullptr) return;
  __shared__ float part[64][33];
  const int cx = threadIdx.x & 3, ry = threadIdx.x >> 2;
  const int64_t c = blockIdx.x * static_cast<int64_t>(32) + cx * 8;  // cols is a multiple of 8
  float s[8] = {};
  if (c < cols) {
#pragma unroll 8
    for (int64_t r = ry; r < rows; r += 64) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(A + r * cols + c));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        s[2 * q] += F16 ? f16_bits_to_f32(w[q] & 0xFFFFu) : bf16_bits_to_f32(w[q] & 0xFFFFu);
        s[2 * q + 1] += F16 ? f16_bits_to_f32(w[q] >> 16) : bf16_bits_to_f32(w[q] >> 16);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) part[ry][cx * 8 + q] = s[q];
  __syncthreads();
  const int64_t oc = blockIdx.x * static_cast<int64_t>(32) + threadIdx.x;
  if (threadIdx.x < 32 && oc < cols) {
    float v = 0.0f;
    for (int r = 0; r < 64; ++r) v += part[r][threadIdx.x];
    out[oc] = static_cast<unsigned short>(pack2_16<OUT>(v, 0.0f));
  }
}

}  // namespace

// Few tiles leave most pairs idle: as many parts of the contraction as keep them busy, of 16
// k-blocks at least. (129 tokens, two sources of 11008 x 4096: 16 tiles; 115 us in one part, 47 in four.)
int dense_splits(int kind, int64_t M, int64_t N, int64_t K, int sources) {
  const int64_t tile_n = kind == kDenseGated ? dense::kBN / 2 : dense::kBN;
  const int64_t tiles = ((M + dense::kBM - 1) / dense::kBM) * ((N + tile_n - 1) / tile_n);
  const int64_t kb = (K + dense::kBK - 1) / dense::kBK * (kind == kDenseBackward ? sources : 1);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kSms / 2 / tiles, kb / 16)));
}

size_t dense_partial_bytes(int kind, int64_t M, int64_t N, int64_t K, int sources) {
  const int splits = dense_splits(kind, M, N, K, sources);
  return splits == 1 ? 0 : static_cast<size_t>(splits) * (kind == kDenseGated ? 2 : 1) * M * N * sizeof(float);
}

cudaError_t launch_dense(const DenseJob& j, cudaStream_t st) {
  return j.x_dtype == kF16 ? launch_dense_kind<true>(j, st) : launch_dense_kind<false>(j, st);
}

cudaError_t read_dense_timeouts(unsigned int* out) {
  return cudaMemcpyFromSymbol(out, g_wait_timeouts, sizeof(unsigned int));
}

cudaError_t launch_gated_grad(const void* dY, const void* G, const void* U, int64_t n, int x_dtype,
                              int act, void* dG, void* dU, cudaStream_t st) {
  if (n == 0) return cudaSuccess;
  return x_dtype == kF16 ? launch_gated_grad_typed<true>(dY, G, U, n, act, dG, dU, st)
                         : launch_gated_grad_typed<false>(dY, G, U, n, act, dG, dU, st);
}

cudaError_t launch_empty_sums(const void* const (&bias)[2], int mats, int64_t M, int64_t N,
                              int x_dtype, int act, void* Y, void* G, void* U, cudaStream_t st) {
  const auto *bg = static_cast<const unsigned short*>(bias[0]),
             *bu = static_cast<const unsigned short*>(bias[1]);
  auto *y = static_cast<unsigned short*>(Y), *g = static_cast<unsigned short*>(G),
       *u = static_cast<unsigned short*>(U);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>((M * N + 255) / 256, 148 * 8));
  if (x_dtype == kF16)
    empty_sums_kernel<true><<<grid, 256, 0, st>>>(bg, bu, mats, M * N, N, act, y, g, u);
  else
    empty_sums_kernel<false><<<grid, 256, 0, st>>>(bg, bu, mats, M * N, N, act, y, g, u);
  return cudaGetLastError();
}

cudaError_t launch_column_sums(const void* A0, void* out0, const void* A1, void* out1, int64_t rows,
                               int64_t cols, int x_dtype, cudaStream_t st) {
  if (cols == 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>((cols + 31) / 32), out1 != nullptr ? 2 : 1);
  const auto *a0 = static_cast<const unsigned short*>(A0), *a1 = static_cast<const unsigned short*>(A1);
  auto *o0 = static_cast<unsigned short*>(out0), *o1 = static_cast<unsigned short*>(out1);
  if (x_dtype == kF16)
    column_sums_kernel<true><<<grid, 256, 0, st>>>(a0, o0, a1, o1, rows, cols);
  else
    column_sums_kernel<false><<<grid, 256, 0, st>>>(a0, o0, a1, o1, rows, cols);
  return cudaGetLastError();
}

}  // namespace hqqk
