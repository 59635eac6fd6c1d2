// hqq_codes.cuh - packed codes of any width to W' in registers: loading, widening, scale and zero,
// with exactly the dequantizer's roundings. Shared by the products that multiply straight from the
// codes. Everything has internal linkage.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "hqq_device.cuh"
#include "hqq_kernels.h"
#include "hqq_tiles.h"

namespace hqqk {
namespace {

// Up to two weights of one format.
struct WeightArgs {
  const uint8_t* packed[2];
  const void* scale[2];
  const void* zero[2];
  const float2* scale_mm[2];
  const float2* zero_mm[2];
  const unsigned short* bias[2];
  int lg_group;   // log2 of the group size
  int meta_dt;    // Dt of scale / zero where they are not 8-bit codes
  int meta_run;   // second-level run length, and its log2 (-1: no power of two)
  int lg_run;
};

// The codes of 32 consecutive elements: 32-bit words, least significant code first (8, 4, 2, 1 bits:
// NBITS words); 3 bits: ten to a word, whose bits 30 and 31 hold anything, as do those past the last.
template <int NBITS>
struct Codes32 {
  static constexpr int kWords = NBITS == 3 ? 4 : NBITS;
  uint32_t w[kWords];
};

// A code is widened by making its bits the mantissa of a half-precision power of two, where they
// stand: at bits 0 .. of a half under 1024 they read 1024 + q, at bits NBITS .. under
// 2^(10 - NBITS) they read that plus q, exactly; one shift serves two masks, and each mask takes two
// codes, 16 bits apart. Pair p of unit u (8 MMA k slots) holds the elements
//   8 bits        8u + 2p, 8u + 2p + 1            2 bits  16(u/2) + 4(u%2) + p, 8 further
//   4 bits        8u + p, 8u + p + 4              1 bit   4u + p, 16 further
// of its chunk of 32, and X is laid out in the same order (slot_element). At 3 bits, codes five apart
// in a word stand 15 bits apart: with the first at bits 1 .. 3, under 512, the second is at bits 0 ..
// 2 of its half, under 1024. Pair i = 4u + p holds 10(i/5) + i%5 and the one 5 further, the last
// pair the last two codes.
template <int NBITS>
__host__ __device__ constexpr int slot_element(int u, int j) {  // slot j = 0 .. 7 of unit u
  const int p = j / 2, h = j % 2;
  return NBITS == 4   ? 8 * u + p + 4 * h
         : NBITS == 2 ? 16 * (u / 2) + 4 * (u % 2) + p + 8 * h
         : NBITS == 1 ? 4 * u + p + 16 * h
         : NBITS == 8 ? 8 * u + j
         : 4 * u + p == 15 ? 30 + h
                           : (4 * u + p) / 5 * 10 + (4 * u + p) % 5 + 5 * h;
}
// (v & mask) | bits in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t bits) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(v), "r"(mask), "r"(bits));
  return d;
}
// Whether a code, the first (h 0) or second of pair p, stands under 1024, and the other base.
template <int NBITS>
__host__ __device__ constexpr bool under_1024(int p, int h) {
  return NBITS == 8 || (NBITS == 3 ? h == 1 : p % 2 == 0);
}
template <int NBITS>
__host__ __device__ constexpr float lesser_base() {
  return NBITS == 8 ? 1024.0f : NBITS == 3 ? 512.0f : static_cast<float>(1 << (10 - NBITS % 8));
}
template <int NBITS>
__device__ __forceinline__ uint32_t widened_pair(const Codes32<NBITS>& c, int u, int p) {
  constexpr uint32_t k1024 = 0x64006400u;
  if constexpr (NBITS == 8) {
    return __byte_perm(c.w[2 * u + p / 2], k1024, p % 2 ? 0x5352 : 0x5150);
  } else if constexpr (NBITS == 3) {
    constexpr uint32_t kBases = 0x64006000u;  // 1024 over 512
    const int i = 4 * u + p, r = i % 5;
    const uint32_t f = c.w[i / 5];
    if (i == 15) return and_or(f << 13, 0x00070000u, and_or(f << 1, 0x0000000Eu, kBases));
    return and_or(r == 0 ? f << 1 : f >> (3 * r - 1), 0x0007000Eu, kBases);
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
// (base + q) - (base + zero) is the one rounding of q - zero (`over_1024`, `over_lesser` alone, by the
// code's base); otherwise the base is subtracted first, exactly, and then zero. Below 2^24 a sum with 1024
// that gives zero back was exact, and the sum with the smaller base is then exact too. From 2^24 on neither
// follows (a bf16 zero of 2^30 swallows a base of 64, one above 2^34 that of 1024, and both come back): such
// zeros take the two steps, as do those next to 0 whose lowest bits a sum with 1024 drops.
struct GroupMeta {
  float scale, over_1024, over_lesser, neg_zero;
};
// What is known of the groups of a chunk: whether every sum with 1024 gave zero back, and the largest zero (one
// comparison for all of them; of fp16 none is needed. A comparison for each: 1 token, 11008 x 4096, 2 bits,
// groups of 32, 15.0 -> 16.1 us; this way 15.0).
struct Exactness {
  bool back = true;
  float most = 0.0f;
  __device__ __forceinline__ bool holds() const { return back && most < 16777216.0f; }
};
template <int NBITS, bool F16>
__device__ __forceinline__ GroupMeta group_meta(float scale, float zero, Exactness* known) {
  const float sum = __fadd_rn(zero, 1024.0f);
  known->back = known->back && __fsub_rn(sum, 1024.0f) == zero;
  if constexpr (!F16) known->most = fmaxf(known->most, fabsf(zero));
  return GroupMeta{scale, -sum, -__fadd_rn(zero, lesser_base<NBITS>()), -zero};
}

// Pair p of unit u as W' in fp32, with the dequantizer's first two roundings: q - zero, * scale. m: the
// chunk's GROUPS groups.
template <int NBITS, int GROUPS, bool ONE>
__device__ __forceinline__ float2 dequant_pair(const Codes32<NBITS>& c, int u, int p,
                                               const GroupMeta* m) {
  const GroupMeta& a = m[slot_element<NBITS>(u, 2 * p) * GROUPS / 32];
  const GroupMeta& b = m[slot_element<NBITS>(u, 2 * p + 1) * GROUPS / 32];
  const uint32_t h = widened_pair<NBITS>(c, u, p);
  float2 v;
  if constexpr (ONE)
    v = add_f32_f16x2(h, make_float2(under_1024<NBITS>(p, 0) ? a.over_1024 : a.over_lesser,
                                     under_1024<NBITS>(p, 1) ? b.over_1024 : b.over_lesser));
  else
    v = fadd2_rn(
        add_f32_f16x2(h, make_float2(under_1024<NBITS>(p, 0) ? -1024.0f : -lesser_base<NBITS>(),
                                     under_1024<NBITS>(p, 1) ? -1024.0f : -lesser_base<NBITS>())),
        make_float2(a.neg_zero, b.neg_zero));
  return fmul2_rn(v, make_float2(a.scale, b.scale));
}

// Unit u of a chunk as W' pairs in slot order, rounded to dt.
template <int NBITS, int OUT, int GROUPS, bool ONE>
__device__ __forceinline__ uint4 dequant_unit(const Codes32<NBITS>& c, int u, const GroupMeta* m) {
  uint32_t o[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float2 v = dequant_pair<NBITS, GROUPS, ONE>(c, u, p, m);
    o[p] = pack2_16<OUT>(v.x, v.y);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// All 32 codes of a chunk as W', in their own order: eight to a uint4.
template <int NBITS, int OUT, int GROUPS, bool ONE>
__device__ __forceinline__ void dequant_chunk(const Codes32<NBITS>& c, const GroupMeta* m,
                                              uint4 (&o)[4]) {
  float2 v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = dequant_pair<NBITS, GROUPS, ONE>(c, i / 4, i % 4, m);
  float e[32];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    e[slot_element<NBITS>(i / 4, 2 * (i % 4))] = v[i].x;
    e[slot_element<NBITS>(i / 4, 2 * (i % 4) + 1)] = v[i].y;
  }
#pragma unroll
  for (int u = 0; u < 4; ++u)
    o[u] = make_uint4(pack2_16<OUT>(e[8 * u], e[8 * u + 1]), pack2_16<OUT>(e[8 * u + 2], e[8 * u + 3]),
                      pack2_16<OUT>(e[8 * u + 4], e[8 * u + 5]),
                      pack2_16<OUT>(e[8 * u + 6], e[8 * u + 7]));
}

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
// 16 bytes, of which the first `bytes` are read and the others become 0.
__device__ __forceinline__ void cp_async_part(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A warp's tile of 16 rows x CODES consecutive codes in shared memory, copied by the warp together:
// neighbouring lanes take neighbouring 16-byte pieces of a row. (Each lane copying its own 32 codes
// touched a sector or two per lane and filled the L1's data path: 32 wavefronts a copy.) The pieces
// of a row are permuted by its number so that reads are free of bank conflicts, for eight lanes that
// read the same piece of eight rows (QUADS false) or chunks 0, 2, 4, 6 of two rows (QUADS true).
// Rows must start on 16-byte boundaries, except at 3 bits, where a row's copy starts at the boundary
// below its first code: pieces of 40 codes, not permuted, the rows an odd number of pieces apart.
template <int NBITS, int CODES, bool QUADS>
struct CodeTile {
  static constexpr int kRow = tile_row_bytes(NBITS, CODES);
  static constexpr int kPiece = kRow < 16 ? kRow : 16;  // not at 3 bits
  static constexpr int kPieces = kRow / kPiece;

  static __device__ __forceinline__ uint32_t place(uint32_t row, uint32_t piece) {
    if constexpr (QUADS && kPieces == 16) return piece ^ ((piece >> 3) & 1) ^ ((row & 1) << 1);
    if constexpr (QUADS) return kPieces == 8 ? piece ^ (row & 1) : piece;
    if constexpr (kPieces > 1) return piece ^ ((row / (8 / kPieces)) & (kPieces - 1));
    return piece;
  }

  // The first `rows` rows and `codes` codes of each. src: the first code's byte, rows `stride` bytes
  // apart; at 3 bits the 16-byte boundary from which `first` counts the first code, rows `stride` codes
  // apart.
  static __device__ __forceinline__ void copy(uint32_t to, const uint8_t* src, uint32_t first,
                                              uint32_t stride, uint32_t rows, uint32_t codes,
                                              uint32_t lane) {
    if constexpr (NBITS == 3) {
      constexpr uint32_t kMost = (39 + CODES - 1) / 40 + 1;  // pieces a row may span
#pragma unroll
      for (uint32_t n = 0; n < (16 * kMost + 31) / 32; ++n) {
        const uint32_t i = n * 32 + lane, row = i / kMost, piece = i - row * kMost;
        const uint32_t e = first + row * stride, p0 = e / 40u;
        // bytes up to the row's last word; nothing further is read
        const int left = static_cast<int>((e - 40u * p0 + codes - 1) / 10u * 4u + 4u - 16u * piece);
        if (row < rows && left > 0)
          cp_async_part(to + row * kRow + piece * 16, src + (p0 + piece) * 16u,
                        static_cast<uint32_t>(min(left, 16)));
      }
    } else {
      constexpr uint32_t kAll = 16 * kPieces;
#pragma unroll
      for (uint32_t n = 0; n < (kAll + 31) / 32; ++n) {
        const uint32_t i = n * 32 + lane, row = i / kPieces, piece = i % kPieces;
        if (i < kAll && row < rows && piece * (kPiece * 8 / NBITS) < codes)
          cp_async<kPiece>(to + row * kRow + place(row, piece) * kPiece,
                           src + row * stride + piece * kPiece);
      }
    }
  }

  // The 32 codes of `row` from code `at` (a multiple of 32) on; at 3 bits, slot: the first code of
  // the row's place in its 16 bytes.
  static __device__ __forceinline__ Codes32<NBITS> read(const uint8_t* tile, uint32_t row, uint32_t at,
                                                        uint32_t slot) {
    Codes32<NBITS> c;
    if constexpr (NBITS == 3) {
      const uint32_t word = (slot + at) / 10u;
      const int first_slot = static_cast<int>(slot + at - 10u * word);
      const uint32_t* p = reinterpret_cast<const uint32_t*>(tile + row * kRow) + word;
      uint32_t v[5];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = p[i];
      v[4] = first_slot == 9 ? p[4] : 0u;  // 31 codes further: the fifth word only from slot 9
      const uint32_t mask = 0x3FFFFFFFu >> (3 * first_slot);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c.w[i] = and_or(v[i] >> (3 * first_slot), mask, v[i + 1] << (30 - 3 * first_slot));
    } else {
      const uint32_t byte = at / 8 * NBITS;
      const uint8_t* line = tile + row * kRow;
      if constexpr (NBITS >= 4) {
#pragma unroll
        for (int i = 0; i < NBITS / 4; ++i) {
          const uint4 v = *reinterpret_cast<const uint4*>(line + place(row, byte / 16 + i) * 16);
          c.w[4 * i] = v.x;
          c.w[4 * i + 1] = v.y;
          c.w[4 * i + 2] = v.z;
          c.w[4 * i + 3] = v.w;
        }
      } else {
        const uint8_t* p = line + place(row, byte / kPiece) * kPiece + byte % kPiece;
        if constexpr (NBITS == 2) {
          const uint2 v = *reinterpret_cast<const uint2*>(p);
          c.w[0] = v.x;
          c.w[1] = v.y;
        } else {
          c.w[0] = *reinterpret_cast<const uint32_t*>(p);
        }
      }
    }
    return c;
  }
};

// Whether rows of `cols` codes can be copied as CodeTile wants them.
inline bool whole_rows(int nbits, int64_t cols) {
  return cols % 32 == 0 && (nbits == 3 || cols / 8 * nbits % 16 == 0);
}

// A lane's chunk straight from memory, for rows of any multiple of 8 codes, in units of 8 codes (NBITS
// bytes, aligned to their size): the first `units` of the chunk exist, the others read as code 0.
template <int NBITS>
__device__ __forceinline__ Codes32<NBITS> load_codes_units(const uint8_t* slab, uint32_t e,
                                                           int units) {
  Codes32<NBITS> c;
#pragma unroll
  for (int i = 0; i < Codes32<NBITS>::kWords; ++i) c.w[i] = 0u;
  uint32_t f[4] = {0u, 0u, 0u, 0u};  // 3 bits: the units
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (u >= units) break;
    if constexpr (NBITS == 3) {
      const uint32_t word = (e + 8u * u) / 10u;
      const int s = static_cast<int>(e + 8u * u - word * 10u);
      const uint32_t* p = reinterpret_cast<const uint32_t*>(slab) + word;
      const uint32_t lo = __ldg(p) & 0x3FFFFFFFu;
      const uint32_t hi = s > 2 ? __ldg(p + 1) : 0u;  // 8 codes from slot 2 end in this word
      f[u] = (lo >> (3 * s) | hi << (30 - 3 * s)) & 0x00FFFFFFu;
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
  if constexpr (NBITS == 3) {
    c.w[0] = f[0] | f[1] << 24;
    c.w[1] = f[1] >> 6 | f[2] << 18;
    c.w[2] = f[2] >> 12 | f[3] << 12;
    c.w[3] = f[3] >> 18;
  }
  return c;
}

// Consecutive rows of one weight: their codes and meta, addressed by 32-bit offsets from here.
struct Slab {
  const uint8_t* codes;   // the first code's byte; at 3 bits the 16-byte boundary below it
  const uint8_t *scale, *zero;
  const float2 *scale_mm, *zero_mm;  // from the run of the slab's first group on, or nullptr
  uint32_t code0;         // 3 bits: the first code's place from there, under 40
  uint32_t group0;        // the first group's place in its run
};

// The slab of the rows from `row` on of matrix i.
template <int NBITS, bool ANY>
__device__ __forceinline__ Slab slab_of_row(const WeightArgs& a, int i, int64_t row, uint32_t K,
                                            uint32_t groups_per_row) {
  const int64_t e0 = row * K, g0 = row * groups_per_row;
  const uint32_t msz = ANY && a.meta_dt == kF32 ? 4 : 2;
  Slab b;
  b.code0 = NBITS == 3 ? static_cast<uint32_t>(e0 % 40) : 0u;
  b.codes = a.packed[i] + (NBITS == 3 ? e0 / 40 * 16 : e0 / 8 * NBITS);
  b.scale_mm = b.zero_mm = nullptr;
  b.group0 = 0;
  if constexpr (ANY) {
    const int64_t run0 = a.lg_run >= 0 ? g0 >> a.lg_run : g0 / a.meta_run;  // (long division is slow)
    b.group0 = static_cast<uint32_t>(g0 - run0 * a.meta_run);
    if (a.scale_mm[i] != nullptr) b.scale_mm = a.scale_mm[i] + run0;
    if (a.zero_mm[i] != nullptr) b.zero_mm = a.zero_mm[i] + run0;
  }
  b.scale = static_cast<const uint8_t*>(a.scale[i]) + g0 * (b.scale_mm != nullptr ? 1 : msz);
  b.zero = static_cast<const uint8_t*>(a.zero[i]) + g0 * (b.zero_mm != nullptr ? 1 : msz);
  return b;
}

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
__device__ __forceinline__ RawMeta<ANY> load_raw_meta(const Slab& b, const WeightArgs& a, uint32_t step,
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

// Groups at and at + 1 of a slab whose scales and zeros are 16-bit values on 4-byte boundaries, the
// second in the upper halves; and one of the two. (Groups of 16, 37 tokens, gated 11008 x 4096: a load for
// each group kept the L1 at 71 % of its rate.)
__device__ __forceinline__ RawMeta<false> load_raw_meta_two(const Slab& b, uint32_t step,
                                                            uint32_t at) {
  return RawMeta<false>{__ldg(reinterpret_cast<const uint32_t*>(b.scale + 2u * step + 2u * at)),
                        __ldg(reinterpret_cast<const uint32_t*>(b.zero + 2u * step + 2u * at))};
}
__device__ __forceinline__ RawMeta<false> one_of_two(const RawMeta<false>& m, int which) {
  return which != 0 ? RawMeta<false>{m.s >> 16, m.z >> 16}
                    : RawMeta<false>{m.s & 0xFFFFu, m.z & 0xFFFFu};
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

// ---------------------------------------------------------------- host side
// Whether some scale or zero is not simply a value of the activation type (RawMeta's ANY).
inline bool any_meta(const WeightView* w, int mats, int meta_dtype, int x_dtype) {
  bool any = meta_dtype != x_dtype;
  for (int i = 0; i < mats; ++i) any = any || w[i].scale_mm != nullptr || w[i].zero_mm != nullptr;
  return any;
}

// Whether groups can be loaded two at a time (load_raw_meta_two); rows then hold an even number.
inline bool meta_by_twos(const WeightView* w, int mats) {
  bool twos = true;
  for (int i = 0; i < mats; ++i)
    twos = twos && (reinterpret_cast<uintptr_t>(w[i].scale) | reinterpret_cast<uintptr_t>(w[i].zero)) % 4 == 0;
  return twos;
}

inline WeightArgs weight_args(const WeightView* w, int mats, int group_size, int meta_dtype,
                              int meta_group_size) {
  WeightArgs a = {};
  for (int i = 0; i < mats; ++i) {
    a.packed[i] = w[i].packed;
    a.scale[i] = w[i].scale;
    a.zero[i] = w[i].zero;
    a.scale_mm[i] = reinterpret_cast<const float2*>(w[i].scale_mm);
    a.zero_mm[i] = reinterpret_cast<const float2*>(w[i].zero_mm);
    a.bias[i] = static_cast<const unsigned short*>(w[i].bias);
  }
  a.lg_group = __builtin_ctz(static_cast<unsigned>(group_size));
  a.meta_dt = meta_dtype;
  a.meta_run = meta_group_size;
  a.lg_run = (meta_group_size & (meta_group_size - 1)) == 0 ? __builtin_ctz(meta_group_size) : -1;
  return a;
}

}  // namespace
}  // namespace hqqk
