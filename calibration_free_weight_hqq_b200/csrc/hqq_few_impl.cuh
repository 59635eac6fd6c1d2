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
//   * Codes come by asynchronous copies several k-blocks ahead (across tiles too), each lane into
//     its own slots (no barrier); scale and zero one k-block ahead in registers.
//   * Lanes without a token of their own (g >= M) repeat the last one; those results are dropped.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "hqq_act.cuh"
#include "hqq_device.cuh"
#include "hqq_few.h"
#include "hqq_kernels.h"
#include "hqq_tensor.cuh"

namespace hqqk {
namespace {

struct FewArgs {
  const uint8_t* packed[2];
  const void* scale[2];
  const void* zero[2];
  const float2* scale_mm[2];
  const float2* zero_mm[2];
  const unsigned short* bias[2];
  const uint8_t* X;
  unsigned short *Y, *G, *U;
  int M, N, K;
  int lg_group;   // log2 of the group size
  int meta_dt;    // Dt of scale / zero where they are not 8-bit codes
  int meta_run;   // second-level run length, and its log2 (-1: no power of two)
  int lg_run;
  int act;
};

// The codes of 32 consecutive elements: 32-bit words, least significant code first (8, 4, 2, 1 bits:
// NBITS words); 3 bits: one 24-bit field of 8 codes per word.
template <int NBITS>
struct Codes32 {
  static constexpr int kWords = NBITS == 3 ? 4 : NBITS;
  uint32_t w[kWords];
};

// A code is widened by making its bits the mantissa of a half-precision power of two, where they
// stand: at bits 0 .. of a half under 1024 they read 1024 + q, at bits NBITS .. under
// 2^(10 - NBITS) they read that plus q, exactly; one shift serves two masks, and each mask takes two
// codes, 16 bits apart. Pair p of unit u (8 MMA k slots) holds the elements
//   8 and 3 bits  8u + 2p, 8u + 2p + 1            2 bits  16(u/2) + 4(u%2) + p, 8 further
//   4 bits        8u + p, 8u + p + 4              1 bit   4u + p, 16 further
// of its chunk of 32, and X is laid out in the same order (few_element).
template <int NBITS>
__host__ __device__ constexpr int few_element(int u, int j) {  // slot j = 0 .. 7 of unit u
  const int p = j / 2, h = j % 2;
  return NBITS == 4   ? 8 * u + p + 4 * h
         : NBITS == 2 ? 16 * (u / 2) + 4 * (u % 2) + p + 8 * h
         : NBITS == 1 ? 4 * u + p + 16 * h
                      : 8 * u + j;
}
// (v & mask) | bits in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t bits) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(v), "r"(mask), "r"(bits));
  return d;
}
// The base under a code of pair p.
template <int NBITS>
__host__ __device__ constexpr float few_base(int p) {
  return NBITS == 8 || NBITS == 3 || p % 2 == 0 ? 1024.0f : static_cast<float>(1 << (10 - NBITS % 8));
}
template <int NBITS>
__device__ __forceinline__ uint32_t widened_pair(const Codes32<NBITS>& c, int u, int p) {
  constexpr uint32_t k1024 = 0x64006400u;
  if constexpr (NBITS == 8) {
    return __byte_perm(c.w[2 * u + p / 2], k1024, p % 2 ? 0x5352 : 0x5150);
  } else if constexpr (NBITS == 3) {
    const uint32_t f = c.w[u];
    const int hi = 6 * p + 3 - 16;  // the second code's way to bit 16
    return and_or(hi < 0 ? f << -hi : f >> hi, 0x00070000u, and_or(f >> (6 * p), 7u, k1024));
  } else {
    constexpr uint32_t kMask = ((1u << NBITS) - 1u) * 0x00010001u;
    constexpr uint32_t kOdd = k1024 - static_cast<uint32_t>(NBITS) * 0x04000400u;  // 2^(10 - NBITS)
    // code j of the pair's word, counted in pairs
    const int j = NBITS == 4 ? p : NBITS == 2 ? 4 * (u % 2) + p : 4 * u + p;
    const uint32_t v = c.w[NBITS == 4 ? u : NBITS == 2 ? u / 2 : 0] >> (NBITS * (j - p % 2));
    return p % 2 ? and_or(v, kMask << NBITS, kOdd) : and_or(v, kMask, k1024);
  }
}

// c + a half-precision value in fp32, rounded once.
__device__ __forceinline__ float2 add_f32_f16x2(uint32_t h, float2 c) {
  float2 d;
  asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "add.rn.f32.f16 %0, lo, %3;\n\tadd.rn.f32.f16 %1, hi, %4;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "r"(h), "f"(c.x), "f"(c.y));
  return d;
}

// A group's scale and zero as the conversion takes them. Where base + zero is exact,
// (base + q) - (base + zero) is the one rounding of q - zero (`even`, `odd` alone, by the pair's
// base); otherwise the base is subtracted first, exactly, and then zero. If 1024 + zero is exact, so
// is the sum with the smaller base. The test is cheap and, for zeros of 8 or 11 significant bits,
// fails only next to 0.
struct GroupMeta {
  float scale, even, odd, neg_zero;
};
template <int NBITS>
__device__ __forceinline__ GroupMeta group_meta(float scale, float zero, bool* one) {
  const float sum = __fadd_rn(zero, 1024.0f);
  *one = *one && __fsub_rn(sum, 1024.0f) == zero;
  return GroupMeta{scale, -sum, -__fadd_rn(zero, few_base<NBITS>(1)), -zero};
}

// Unit u of a chunk as W' pairs, with the dequantizer's three roundings: q - zero, * scale, to dt.
// m: the chunk's GROUPS groups.
template <int NBITS, int OUT, int GROUPS, bool ONE>
__device__ __forceinline__ uint4 dequant_unit(const Codes32<NBITS>& c, int u, const GroupMeta* m) {
  uint32_t o[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const GroupMeta& a = m[few_element<NBITS>(u, 2 * p) * GROUPS / 32];
    const GroupMeta& b = m[few_element<NBITS>(u, 2 * p + 1) * GROUPS / 32];
    const uint32_t h = widened_pair<NBITS>(c, u, p);
    float2 v;
    if constexpr (ONE)
      v = add_f32_f16x2(h, p % 2 ? make_float2(a.odd, b.odd) : make_float2(a.even, b.even));
    else
      v = fadd2_rn(add_f32_f16x2(h, make_float2(-few_base<NBITS>(p), -few_base<NBITS>(p))),
                   make_float2(a.neg_zero, b.neg_zero));
    v = fmul2_rn(v, make_float2(a.scale, b.scale));
    o[p] = pack2_16<OUT>(v.x, v.y);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Copies through L1: a lane's 32 contiguous bytes are one sector in two pieces, and bypassing L1 would
// fetch it twice (28672 x 4096, one token: 32 -> 28 us).
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global.L2::128B [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Copies a lane's 32 codes into its own shared-memory slot: from byte `off` of `base` on or, at
// 3 bits, from element `off` on counted from the first code of the word at `base`. Row lengths are
// multiples of 32 codes, so every copy is aligned to its width. A slot's pieces lie 32 lanes apart, so
// that a warp's pieces are contiguous. `slot` points at the lane's first piece.
template <int NBITS>
__device__ __forceinline__ void copy_chunk(uint32_t slot, const uint8_t* base, uint32_t off) {
  if constexpr (NBITS == 3) {
    const uint32_t word = off / 10u, first = off - word * 10u;
    const uint8_t* p = base + word * 4u;
#pragma unroll
    for (int i = 0; i < 5; ++i)  // 31 codes further: the fifth word only from slot 9
      if (i < 4 || first == 9u) cp_async<4>(slot + i * 128, p + 4 * i);
  } else {
    constexpr int kPiece = NBITS >= 4 ? 16 : 4 * NBITS;
#pragma unroll
    for (int i = 0; i < 4 * NBITS / kPiece; ++i)
      cp_async<kPiece>(slot + i * 32 * kPiece, base + off + i * kPiece);
  }
}

// The chunk in a lane's slot (3 bits: `off` as it was copied).
template <int NBITS>
__device__ __forceinline__ Codes32<NBITS> read_chunk(const uint8_t* slot, uint32_t off) {
  Codes32<NBITS> c;
  if constexpr (NBITS == 3) {
    uint32_t v[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) v[i] = *reinterpret_cast<const uint32_t*>(slot + 128 * i);
    const int first_slot = static_cast<int>(off % 10u);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int at = first_slot + 8 * u;      // 8u .. 8u + 9
      const int first = 8 * u / 10;           // the word of code 8u, or the next one
      const bool next = at >= 10 * (first + 1);
      const int s = at - 10 * (first + (next ? 1 : 0));
      const uint32_t lo = next ? v[first + 1] : v[first];
      const uint32_t hi = next ? v[first + 2 < 5 ? first + 2 : 4] : v[first + 1];
      c.w[u] = (lo & 0x3FFFFFFFu) >> (3 * s) | hi << (30 - 3 * s);
    }
  } else if constexpr (NBITS >= 4) {
#pragma unroll
    for (int i = 0; i < NBITS / 4; ++i) {
      const uint4 v = *reinterpret_cast<const uint4*>(slot + 512 * i);
      c.w[4 * i] = v.x;
      c.w[4 * i + 1] = v.y;
      c.w[4 * i + 2] = v.z;
      c.w[4 * i + 3] = v.w;
    }
  } else if constexpr (NBITS == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(slot);
    c.w[0] = v.x;
    c.w[1] = v.y;
  } else {
    c.w[0] = *reinterpret_cast<const uint32_t*>(slot);
  }
  return c;
}

// As above for rows of any multiple of 8 codes, in units of 8 codes (NBITS bytes, aligned to their
// size): the first `units` of the chunk exist, the others read as code 0.
template <int NBITS>
__device__ __forceinline__ Codes32<NBITS> load_codes_units(const uint8_t* slab, uint32_t e,
                                                           int units) {
  Codes32<NBITS> c;
#pragma unroll
  for (int i = 0; i < Codes32<NBITS>::kWords; ++i) c.w[i] = 0u;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (u >= units) break;
    if constexpr (NBITS == 3) {
      const uint32_t word = (e + 8u * u) / 10u;
      const int s = static_cast<int>(e + 8u * u - word * 10u);
      const uint32_t* p = reinterpret_cast<const uint32_t*>(slab) + word;
      const uint32_t lo = __ldg(p) & 0x3FFFFFFFu;
      const uint32_t hi = s > 2 ? __ldg(p + 1) : 0u;  // 8 codes from slot 2 end in this word
      c.w[u] = lo >> (3 * s) | hi << (30 - 3 * s);
    } else {
      const uint8_t* p = slab + static_cast<uint64_t>((e / 8u + u) * NBITS);
      if constexpr (NBITS == 8) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
        c.w[2 * u] = v.x;
        c.w[2 * u + 1] = v.y;
      } else if constexpr (NBITS == 4) {
        c.w[u] = __ldg(reinterpret_cast<const uint32_t*>(p));
      } else if constexpr (NBITS == 2) {
        c.w[u / 2] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(p)))
                      << (16 * (u % 2));
      } else {
        c.w[0] |= static_cast<uint32_t>(__ldg(p)) << (8 * u);
      }
    }
  }
  return c;
}

// A CTA's part of one weight: its 16 rows' codes and meta.
struct Slab {
  const uint8_t* codes;   // see copy_chunk
  const uint8_t *scale, *zero;
  const float2 *scale_mm, *zero_mm;  // from the run of the slab's first group on, or nullptr
  uint32_t code0;         // 3 bits: slot of the slab's first code in its word
  uint32_t group0;        // the first group's place in its run
};

// Scale and zero of a group as loaded. ANY false: 16-bit values of the activation type. ANY true:
// values of any meta type, or 8-bit codes with their run's (step2, zero2).
template <bool ANY>
struct RawMeta {
  uint32_t s, z;
};
template <>
struct RawMeta<true> {
  uint32_t s, z;
  float2 sp, zp;
};

__device__ __forceinline__ uint32_t load_meta_bits(const uint8_t* p, int dt, bool code, uint32_t i) {
  if (code) return __ldg(p + i);
  if (dt == kF32) return __ldg(reinterpret_cast<const uint32_t*>(p) + i);
  return __ldg(reinterpret_cast<const unsigned short*>(p) + i);
}
__device__ __forceinline__ float meta_value(uint32_t b, int dt) {
  return dt == kF32 ? __uint_as_float(b) : dt == kBF16 ? bf16_bits_to_f32(b) : f16_bits_to_f32(b);
}

// Group `step + at` of a slab (`step` uniform over the warp).
template <bool ANY>
__device__ __forceinline__ RawMeta<ANY> load_raw_meta(const Slab& b, const FewArgs& a, uint32_t step,
                                                      uint32_t at) {
  RawMeta<ANY> m;
  if constexpr (ANY) {
    const uint32_t i = step + at, in = b.group0 + i;
    const uint32_t run = a.lg_run >= 0 ? in >> a.lg_run : in / static_cast<uint32_t>(a.meta_run);
    m.sp = b.scale_mm != nullptr ? __ldg(b.scale_mm + run) : make_float2(0.0f, 0.0f);
    m.zp = b.zero_mm != nullptr ? __ldg(b.zero_mm + run) : make_float2(0.0f, 0.0f);
    m.s = load_meta_bits(b.scale, a.meta_dt, b.scale_mm != nullptr, i);
    m.z = load_meta_bits(b.zero, a.meta_dt, b.zero_mm != nullptr, i);
  } else {
    m.s = __ldg(reinterpret_cast<const unsigned short*>(b.scale + 2u * step + 2u * at));
    m.z = __ldg(reinterpret_cast<const unsigned short*>(b.zero + 2u * step + 2u * at));
  }
  return m;
}

// (scale, zero) in fp32; 8-bit codes are rebuilt as (code - zero2) * step2.
template <bool ANY, bool F16>
__device__ __forceinline__ float2 meta_f32_pair(const RawMeta<ANY>& m, const Slab& b, int dt) {
  if constexpr (ANY) {
    const float s = b.scale_mm != nullptr
                        ? __fmul_rn(__fsub_rn(static_cast<float>(m.s), m.sp.y), m.sp.x)
                        : meta_value(m.s, dt);
    const float z = b.zero_mm != nullptr
                        ? __fmul_rn(__fsub_rn(static_cast<float>(m.z), m.zp.y), m.zp.x)
                        : meta_value(m.z, dt);
    return make_float2(s, z);
  } else {
    return F16 ? make_float2(f16_bits_to_f32(m.s), f16_bits_to_f32(m.z))
               : make_float2(bf16_bits_to_f32(m.s), bf16_bits_to_f32(m.z));
  }
}

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
// in few_element's order, at piece 4p + t. Rows are padded by four pieces, so that 8 lanes - two
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
        const int a = few_element<NBITS>(u, 2 * q), b = few_element<NBITS>(u, 2 * q + 1);
        o[q] = __byte_perm(v[a / 2], v[b / 2], (a % 2 ? 0x32 : 0x10) | (b % 2 ? 0x7600 : 0x5400));
      }
      dst[4 * u] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// GROUP: 64 (groups of 64 codes or more), 32, 16 (K a multiple of 32 with both) or 8 (any group size
// and K; codes and meta read where they are used). ANY: see RawMeta.
template <int NBITS, bool F16, int MATS, int GROUP, bool ANY>
__global__ void __launch_bounds__(32 * kFewMaxWarps, 1) few_tokens_kernel(const FewArgs a) {
  constexpr int OUT = F16 ? kF16 : kBF16;
  constexpr bool kWhole = GROUP != 8;
  constexpr int kGroups = 64 / GROUP;            // groups of a lane's codes of a k-block
  constexpr int kGroupsHalf = kGroups > 1 ? kGroups / 2 : 1;
  constexpr int kDepth = few_depth(NBITS, MATS);
  constexpr int kSlot = 32 * few_chunk(NBITS);   // a warp's chunks of 8 rows
  constexpr int kPiece = NBITS == 3 ? 4 : NBITS >= 4 ? 16 : 4 * NBITS;
  extern __shared__ __align__(16) uint8_t smem[];
  // the shuffle tells the compiler that a warp's index, and all that follows from it, is uniform
  const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);
  const uint32_t warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  const uint32_t g = lane >> 2, t = lane & 3;
  const uint32_t K = static_cast<uint32_t>(a.K), KB = (K + kFewKB - 1) / kFewKB;
  const uint32_t groups_per_row = K >> a.lg_group;
  const uint32_t tiles = (static_cast<uint32_t>(a.N) + kFewRows - 1) / kFewRows;
  uint4* xs = reinterpret_cast<uint4*>(smem);
  uint8_t* after_x = smem + static_cast<size_t>(a.M) * few_x_row(K);
  float* red = reinterpret_cast<float*>(after_x);  // [MATS][warps][8][kFewRedStride]
  uint8_t* ring = after_x + MATS * warps * kFewRed + warp * (kDepth * 2 * MATS * 2 * kSlot) +
                  lane * kPiece;
  const uint32_t ring_u = smem_u32(ring);

  // Rows g and g + 8 of a tile. N is a multiple of 8: rows 8 .. 15 all exist or none does, and where
  // they do not (the last tile), rows 0 .. 7 are read in their place and the results dropped.
  auto second_row = [&](uint32_t tile) {
    return tile * kFewRows + 8 < static_cast<uint32_t>(a.N) ? g + 8 : g;
  };
  const uint32_t msz = ANY && a.meta_dt == kF32 ? 4 : 2;
  auto make_slab = [&](int i, uint32_t tile) {
    const int64_t n0 = static_cast<int64_t>(tile) * kFewRows;
    const int64_t e0 = n0 * a.K, g0 = n0 * groups_per_row;
    Slab b;
    b.code0 = NBITS == 3 ? static_cast<uint32_t>(e0 % 10) : 0u;
    b.codes = a.packed[i] + (NBITS == 3 ? e0 / 10 * 4 : e0 / 8 * NBITS);
    b.scale_mm = b.zero_mm = nullptr;
    b.group0 = 0;
    if constexpr (ANY) {
      const int64_t run0 = g0 / a.meta_run;
      b.group0 = static_cast<uint32_t>(g0 - run0 * a.meta_run);
      if (a.scale_mm[i] != nullptr) b.scale_mm = a.scale_mm[i] + run0;
      if (a.zero_mm[i] != nullptr) b.zero_mm = a.zero_mm[i] + run0;
    }
    b.scale = static_cast<const uint8_t*>(a.scale[i]) + g0 * (b.scale_mm != nullptr ? 1 : msz);
    b.zero = static_cast<const uint8_t*>(a.zero[i]) + g0 * (b.zero_mm != nullptr ? 1 : msz);
    return b;
  };

  // --- codes, kDepth k-blocks ahead: (copy_tile, copy_kb) is the next to ask for. A lane's place in
  // a tile (copy_at) and a k-block's (uniform) add up to its address.
  constexpr uint32_t kStepCodes = NBITS == 3 ? kFewKB : kFewKB / 8 * NBITS;
  auto lane_codes = [&](uint32_t row) {
    const uint32_t e = row * K + 64 * t;
    return NBITS == 3 ? e : e / 8 * NBITS;
  };
  uint32_t copy_tile = warp < KB ? blockIdx.x : tiles, copy_kb = warp;
  const uint8_t* copy_base[MATS];
  uint32_t copy_code0[MATS];
  uint32_t copy_at[2] = {lane_codes(g), 0};
  auto aim_copies = [&]() {
    if (copy_tile < tiles) {
#pragma unroll
      for (int i = 0; i < MATS; ++i) {
        const Slab b = make_slab(i, copy_tile);
        copy_base[i] = b.codes;
        copy_code0[i] = b.code0;
      }
      copy_at[1] = lane_codes(second_row(copy_tile));
    }
  };
  auto copy_half = [&](uint32_t st, int h) {
    if (copy_tile < tiles) {
      // a whole k-block, or the lane's chunk of a partial one
      if ((copy_kb + 1) * kFewKB <= K || copy_kb * kFewKB + 64 * t + 32 * h < K) {
#pragma unroll
        for (int i = 0; i < MATS; ++i) {
          const uint32_t step = copy_kb * kStepCodes + h * (kStepCodes / 8);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t slot = ring_u + (((st * 2 + h) * MATS + i) * 2 + r) * kSlot;
            if constexpr (NBITS == 3)
              copy_chunk<NBITS>(slot, copy_base[i], copy_code0[i] + step + copy_at[r]);
            else
              copy_chunk<NBITS>(slot, copy_base[i] + step, copy_at[r]);
          }
        }
      }
    }
    cp_async_commit();
  };
  auto next_copy = [&]() {
    copy_kb += warps;
    if (copy_kb >= KB && copy_tile < tiles) {
      copy_kb = warp;
      copy_tile += gridDim.x;
      aim_copies();
    }
  };
  if constexpr (kWhole) {
    aim_copies();
#pragma unroll 1
    for (uint32_t s = 0; s < kDepth; ++s) {
      copy_half(s, 0);
      copy_half(s, 1);
      next_copy();
    }
  }

  stage_x<NBITS>(xs, a.X, static_cast<uint32_t>(a.M), K, KB);
  __syncthreads();
  const uint4* xrow = xs + min(g, static_cast<uint32_t>(a.M) - 1) * (few_x_row(K) / 16) + t;

  // --- scale and zero, one k-block ahead. A k-block is a whole number of groups, so a lane's place
  // in a tile and a k-block's (uniform) add up here too.
  Slab slab[MATS];
  uint32_t row1 = g;
  uint32_t meta_at[2] = {g * groups_per_row + ((64 * t) >> a.lg_group), 0};
  RawMeta<ANY> next[MATS][2][kGroups];
  auto aim = [&](uint32_t tile) {
#pragma unroll
    for (int i = 0; i < MATS; ++i) slab[i] = make_slab(i, tile);
    row1 = second_row(tile);
    meta_at[1] = row1 * groups_per_row + ((64 * t) >> a.lg_group);
  };
  auto fetch_meta = [&](uint32_t kb) {
    const uint32_t step = (kb * kFewKB) >> a.lg_group;
    const bool whole = (kb + 1) * kFewKB <= K;
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
      if (!whole && kb * kFewKB + 64 * t + GROUP * u >= K) break;
#pragma unroll
      for (int i = 0; i < MATS; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          next[i][r][u] = load_raw_meta<ANY>(slab[i], a, step, meta_at[r] + u);
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
        bool one = !ANY;
#pragma unroll
        for (int i = 0; i < MATS; ++i)
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int u = 0; u < kGroups; ++u) {
              float2 sz = meta_f32_pair<ANY, F16>(next[i][r][u], slab[i], a.meta_dt);
              if (tail && kb * kFewKB + 64 * t + GROUP * u >= K)
                sz = make_float2(0.0f, 0.0f);  // W' = 0 past K
              m[i][r][u] = group_meta<NBITS>(sz.x, sz.y, &one);
            }
        one = !ANY && __all_sync(0xFFFFFFFFu, one);
        uint32_t off[MATS][2];  // 3 bits: where the chunks start in their words
#pragma unroll
        for (int i = 0; i < MATS; ++i) {
          off[i][0] = slab[i].code0 + g * K + kb * kFewKB + 64 * t;
          off[i][1] = slab[i].code0 + row1 * K + kb * kFewKB + 64 * t;
        }
        // the next k-block's meta, of the next tile after this one's last
        if (kb + warps < KB) {
          fetch_meta(kb + warps);
        } else if (tile + gridDim.x < tiles) {
          aim(tile + gridDim.x);
          fetch_meta(warp);
        }
        const uint8_t* slots = ring + st * (2 * MATS * 2 * kSlot);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          cp_async_wait<2 * kDepth - 1>();  // the lane's own copies: no other thread reads them
#pragma unroll
          for (int i = 0; i < MATS; ++i) {
            Codes32<NBITS> c[2];
#pragma unroll
            for (int r = 0; r < 2; ++r)
              c[r] = read_chunk<NBITS>(slots + ((h * MATS + i) * 2 + r) * kSlot, off[i][r] + 32 * h);
            const GroupMeta* m0 = m[i][0] + (kGroups > 1 ? h * kGroupsHalf : 0);
            const GroupMeta* m1 = m[i][1] + (kGroups > 1 ? h * kGroupsHalf : 0);
            if (one)
              multiply_chunk<NBITS, F16, kGroupsHalf, true>(acc[i], c, m0, m1, x + 16 * h);
            else
              multiply_chunk<NBITS, F16, kGroupsHalf, false>(acc[i], c, m0, m1, x + 16 * h);
          }
          copy_half(st, h);  // into the slots just read
        }
        next_copy();
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
            bool one = false;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint32_t row = r == 0 ? g : row1;
              c[r] = load_codes_units<NBITS>(slab[i].codes, slab[i].code0 + row * K + kh, units);
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                float2 sz = make_float2(0.0f, 0.0f);
                if (u < units)
                  sz = meta_f32_pair<ANY, F16>(
                      load_raw_meta<ANY>(slab[i], a, 0u,
                                         row * groups_per_row + ((kh + 8 * u) >> a.lg_group)),
                      slab[i], a.meta_dt);
                m[r][u] = group_meta<NBITS>(sz.x, sz.y, &one);
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
        if (a.bias[i] != nullptr) {
          const uint32_t b = a.bias[i][n];
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
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(tiles, 148 * (16 / warps)));
  const size_t smem = few_smem(NBITS, MATS, warps, j.M, j.K);
  bool any = j.meta_dtype != j.x_dtype;
  for (int i = 0; i < MATS; ++i)
    any = any || a.scale_mm[i] != nullptr || a.zero_mm[i] != nullptr;
  const bool whole = j.K % 32 == 0;
  auto kernel = few_tokens_kernel<NBITS, F16, MATS, 8, true>;
  if (j.group_size >= 64)
    kernel = any ? few_tokens_kernel<NBITS, F16, MATS, 64, true>
                 : few_tokens_kernel<NBITS, F16, MATS, 64, false>;
  else if (j.group_size == 32)
    kernel = any ? few_tokens_kernel<NBITS, F16, MATS, 32, true>
                 : few_tokens_kernel<NBITS, F16, MATS, 32, false>;
  else if (whole && j.group_size == 16 && !any)
    kernel = few_tokens_kernel<NBITS, F16, MATS, 16, false>;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
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
  for (int i = 0; i < j.mats; ++i) {
    a.packed[i] = j.w[i].packed;
    a.scale[i] = j.w[i].scale;
    a.zero[i] = j.w[i].zero;
    a.scale_mm[i] = reinterpret_cast<const float2*>(j.w[i].scale_mm);
    a.zero_mm[i] = reinterpret_cast<const float2*>(j.w[i].zero_mm);
    a.bias[i] = static_cast<const unsigned short*>(j.w[i].bias);
  }
  a.X = static_cast<const uint8_t*>(j.X);
  a.Y = static_cast<unsigned short*>(j.Y);
  a.G = static_cast<unsigned short*>(j.G);
  a.U = static_cast<unsigned short*>(j.U);
  a.M = static_cast<int>(j.M);
  a.N = static_cast<int>(j.N);
  a.K = static_cast<int>(j.K);
  a.lg_group = __builtin_ctz(static_cast<unsigned>(j.group_size));
  a.meta_dt = j.meta_dtype;
  a.meta_run = j.meta_group_size;
  a.lg_run = (a.meta_run & (a.meta_run - 1)) == 0 ? __builtin_ctz(a.meta_run) : -1;
  a.act = j.act;
  const bool f16 = j.x_dtype == kF16;
  if (j.mats == 1)
    return f16 ? launch_few_typed<NBITS, true, 1>(j, a, st)
               : launch_few_typed<NBITS, false, 1>(j, a, st);
  return f16 ? launch_few_typed<NBITS, true, 2>(j, a, st)
             : launch_few_typed<NBITS, false, 2>(j, a, st);
}

}  // namespace hqqk
