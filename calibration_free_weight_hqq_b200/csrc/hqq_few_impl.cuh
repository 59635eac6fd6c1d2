// hqq_few_impl.cuh - products of a few tokens with quantized weights of any format (axis 1).
//
// Y[m, n] = dt( sum_k X[m, k] W'[n, k] + bias[n] ), W' = dt((code - zero) * scale) exactly as the
// dequantizer writes it, fp32 accumulation; with two weights (the gated pair)
// Y = dt( act(X Wg'^T + bg) * (X Wu'^T + bu) ), both projections in one pass over X.
//
// With few tokens the packed weight is read once and the work is its conversion. Each warp
// converts codes in registers straight into the A fragments of the warp-level MMA
// (mma.sync m16n8k16, fp32 accumulators): 16 weight rows are its M, 8 tokens its N, so a
// converted fragment serves every token tile and nothing passes through shared memory.
//   * k-blocks of 128: lane (g, t) = (lane / 4, lane % 4) takes the 32 consecutive codes
//     k = 32t .. 32t+31 of rows g and g + 8 (nbits * 4 bytes each, up to 16-byte loads), and of X
//     the same 32 values of token g. The contraction order inside a k-block is permuted the same
//     way on both operands: MMA step s takes k = 32t + 4s + {0, 1, 2, 3} at the k slots
//     {2t, 2t+1, 2t+8, 2t+9} which lane t holds.
//   * The warps of a CTA share 16 rows and split K, k-block by k-block in turn; their partial
//     sums meet in shared memory and are added in warp order (deterministic).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "hqq_act.cuh"
#include "hqq_device.cuh"
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
  int meta_run;   // second-level run length
  int act;
};

constexpr int kFewWarps = 8;
constexpr int kFewRows = 16;     // weight rows per CTA
constexpr int kFewKB = 128;      // codes of a row per k-block
constexpr int kFewStages = 2;    // k-blocks whose codes are in flight per warp
constexpr int kFewRedStride = kFewRows + 4;  // floats per token of a partial tile: the stores
                                             // of a fragment fall on 32 different banks

// The raw codes of 32 consecutive elements: 32-bit words, least significant code first (8, 4, 2,
// 1 bits: NBITS words); 3 bits: one 24-bit field of 8 codes per word.
template <int NBITS>
struct Codes32 {
  static constexpr int kWords = NBITS == 3 ? 4 : NBITS;
  uint32_t w[kWords];
};

// fp32 2^23 + code j (compile-time j) of a chunk.
template <int NBITS>
__device__ __forceinline__ float magic_code(const Codes32<NBITS>& c, int j) {
  constexpr uint32_t kExp = 0x4B000000u;
  if constexpr (NBITS == 8) {
    return __uint_as_float(__byte_perm(c.w[j / 4], kExp, 0x7540 + j % 4));
  } else if constexpr (NBITS == 4) {
    const uint32_t b = (j & 1) ? (c.w[j / 8] >> 4) & 0x0F0F0F0Fu : c.w[j / 8] & 0x0F0F0F0Fu;
    return __uint_as_float(__byte_perm(b, kExp, 0x7540 + (j % 8) / 2));
  } else if constexpr (NBITS == 2) {
    const uint32_t b = (c.w[j / 16] >> (2 * (j % 4))) & 0x03030303u;
    return __uint_as_float(__byte_perm(b, kExp, 0x7540 + (j % 16) / 4));
  } else if constexpr (NBITS == 1) {
    const uint32_t b = (c.w[0] >> (j % 8)) & 0x01010101u;
    return __uint_as_float(__byte_perm(b, kExp, 0x7540 + j / 8));
  } else {
    return __uint_as_float(((c.w[j / 8] >> (3 * (j % 8))) & 7u) | kExp);
  }
}

// Codes 8u .. 8u+7 of a chunk as W' pairs: (2^23 + q) - 2^23 is exact, then the dequantizer's
// three roundings (q - zero, * scale, to dt), on fp32 pairs.
template <int NBITS, int OUT>
__device__ __forceinline__ uint4 dequant_unit(const Codes32<NBITS>& c, int u, float neg_zero,
                                              float scale) {
  const float2 neg_magic = make_float2(-8388608.0f, -8388608.0f);
  const float2 nz = make_float2(neg_zero, neg_zero), sc = make_float2(scale, scale);
  uint32_t o[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float2 m = make_float2(magic_code<NBITS>(c, 8 * u + 2 * p),
                                 magic_code<NBITS>(c, 8 * u + 2 * p + 1));
    const float2 v = fmul2_rn(fadd2_rn(fadd2_rn(m, neg_magic), nz), sc);
    o[p] = pack2_16<OUT>(v.x, v.y);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ uint4 ld_stream16(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// The 32 codes of row `row` from column k on (k a multiple of 32, K a multiple of 32: every load
// is aligned to its width).
template <int NBITS>
__device__ __forceinline__ void load_codes_whole(Codes32<NBITS>& c, const uint8_t* packed,
                                                 int64_t row, int k, int K) {
  if constexpr (NBITS == 3) {
    const int64_t e = row * K + k;
    const int64_t word = e / 10;
    const int slot = static_cast<int>(e - word * 10);
    const uint32_t* p = reinterpret_cast<const uint32_t*>(packed) + word;
    uint32_t v[5];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __ldg(p + i);
    v[4] = slot == 9 ? __ldg(p + 4) : 0u;  // 31 codes further: the fifth word only from slot 9
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int at = slot + 8 * u;            // 8u .. 8u + 9
      const int first = 8 * u / 10;           // the word of code 8u, or the next one
      const bool next = at >= 10 * (first + 1);
      const int s = at - 10 * (first + (next ? 1 : 0));
      const uint32_t lo = next ? v[first + 1] : v[first];
      const uint32_t hi = next ? v[first + 2 < 5 ? first + 2 : 4] : v[first + 1];
      c.w[u] = (lo & 0x3FFFFFFFu) >> (3 * s) | hi << (30 - 3 * s);
    }
  } else {
    const uint8_t* p = packed + (row * K + k) / 8 * NBITS;
    if constexpr (NBITS >= 4) {
#pragma unroll
      for (int i = 0; i < NBITS / 4; ++i) {
        const uint4 v = ld_stream16(p + 16 * i);
        c.w[4 * i] = v.x;
        c.w[4 * i + 1] = v.y;
        c.w[4 * i + 2] = v.z;
        c.w[4 * i + 3] = v.w;
      }
    } else if constexpr (NBITS == 2) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
      c.w[0] = v.x;
      c.w[1] = v.y;
    } else {
      c.w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    }
  }
}

// As above for any K that is a multiple of 8, in units of 8 codes (NBITS bytes, aligned to their
// size): the first `units` of the chunk exist, the others read as code 0.
template <int NBITS>
__device__ __forceinline__ void load_codes_units(Codes32<NBITS>& c, const uint8_t* packed,
                                                 int64_t row, int k, int K, int units) {
#pragma unroll
  for (int i = 0; i < Codes32<NBITS>::kWords; ++i) c.w[i] = 0u;
  const int64_t e = row * K + k;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (u >= units) break;
    if constexpr (NBITS == 3) {
      const int64_t word = (e + 8 * u) / 10;
      const int s = static_cast<int>(e + 8 * u - word * 10);
      const uint32_t* p = reinterpret_cast<const uint32_t*>(packed) + word;
      const uint32_t lo = __ldg(p) & 0x3FFFFFFFu;
      const uint32_t hi = s > 2 ? __ldg(p + 1) : 0u;  // 8 codes from slot 2 end in this word
      c.w[u] = lo >> (3 * s) | hi << (30 - 3 * s);
    } else {
      const uint8_t* p = packed + (e / 8 + u) * NBITS;
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
}

// Scale and zero of group i of matrix `mat`, in fp32. MM: either may be 8-bit codes of a second
// level, rebuilt as (code - zero2) * step2.
struct Meta {
  float scale, neg_zero;
};
template <bool MM>
__device__ __forceinline__ Meta load_group_meta(const FewArgs& a, int mat, int64_t i) {
  Meta m;
  if constexpr (MM) {
    const int64_t run = i / a.meta_run;
    if (a.scale_mm[mat] != nullptr) {
      const float2 p = __ldg(a.scale_mm[mat] + run);
      const float q = static_cast<float>(__ldg(static_cast<const uint8_t*>(a.scale[mat]) + i));
      m.scale = __fmul_rn(__fsub_rn(q, p.y), p.x);
    } else {
      m.scale = load_meta(a.scale[mat], a.meta_dt, i);
    }
    if (a.zero_mm[mat] != nullptr) {
      const float2 p = __ldg(a.zero_mm[mat] + run);
      const float q = static_cast<float>(__ldg(static_cast<const uint8_t*>(a.zero[mat]) + i));
      m.neg_zero = -__fmul_rn(__fsub_rn(q, p.y), p.x);
    } else {
      m.neg_zero = -load_meta(a.zero[mat], a.meta_dt, i);
    }
  } else {
    m.scale = load_meta(a.scale[mat], a.meta_dt, i);
    m.neg_zero = -load_meta(a.zero[mat], a.meta_dt, i);
  }
  return m;
}

// GROUP: 32 (groups of 32 or more codes, K a multiple of 32), 16 (groups of 16, K a multiple of
// 32) or 8 (any group size and K). NT: token tiles of 8.
template <int NBITS, bool F16, int NT, int MATS, int GROUP, bool MM>
__global__ void __launch_bounds__(32 * kFewWarps, 2) few_tokens_kernel(const FewArgs a) {
  constexpr int OUT = F16 ? kF16 : kBF16;
  constexpr bool kWhole = GROUP != 8;
  constexpr int kGroups = 32 / GROUP;  // groups of a lane's chunk
  __shared__ float red[MATS][kFewWarps][NT * 8 * kFewRedStride];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * kFewRows, tok0 = blockIdx.y * (8 * NT);
  const int KB = (a.K + kFewKB - 1) / kFewKB;
  const int64_t groups_per_row = a.K >> a.lg_group;

  float acc[MATS][NT][4];
#pragma unroll
  for (int i = 0; i < MATS; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[i][j][q] = 0.0f;

  Codes32<NBITS> codes[kFewStages][MATS][2];
  Meta meta[kFewStages][MATS][2][kGroups];
  auto fetch = [&](int st, int kb) {
    const int k = kb * kFewKB + 32 * t;
    const int left = a.K - k;  // a multiple of 8; of 32 when kWhole
#pragma unroll
    for (int i = 0; i < MATS; ++i) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int64_t row = n0 + g + 8 * r;
        const bool in = row < a.N && left > 0;
        if (in) {
          if constexpr (kWhole)
            load_codes_whole<NBITS>(codes[st][i][r], a.packed[i], row, k, a.K);
          else
            load_codes_units<NBITS>(codes[st][i][r], a.packed[i], row, k, a.K, left >> 3);
        } else {
#pragma unroll
          for (int q = 0; q < Codes32<NBITS>::kWords; ++q) codes[st][i][r].w[q] = 0u;
        }
#pragma unroll
        for (int u = 0; u < kGroups; ++u) {
          // where nothing is read, scale 0 and zero 0 make W' = 0
          const bool have = in && (kWhole || 8 * u < left);
          const int64_t gi = row * groups_per_row + ((k + GROUP * u) >> a.lg_group);
          meta[st][i][r][u] = have ? load_group_meta<MM>(a, i, gi) : Meta{0.0f, 0.0f};
        }
      }
    }
  };

#pragma unroll
  for (int st = 0; st < kFewStages; ++st)
    if (warp + st * kFewWarps < KB) fetch(st, warp + st * kFewWarps);

  for (int kb0 = warp; kb0 < KB; kb0 += kFewWarps * kFewStages) {
#pragma unroll
    for (int st = 0; st < kFewStages; ++st) {
      const int kb = kb0 + st * kFewWarps;
      if (kb >= KB) break;
      // X: 32 values of token tok0 + 8j + g from k on (zero past M and past K)
      uint32_t x[NT][16];
      const int k = kb * kFewKB + 32 * t;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int tok = tok0 + 8 * j + g;
        const uint8_t* p = a.X + (static_cast<int64_t>(tok) * a.K + k) * 2;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (tok < a.M && k + 8 * u < a.K) v = __ldg(reinterpret_cast<const uint4*>(p) + u);
          x[j][4 * u] = v.x;
          x[j][4 * u + 1] = v.y;
          x[j][4 * u + 2] = v.z;
          x[j][4 * u + 3] = v.w;
        }
      }
#pragma unroll
      for (int i = 0; i < MATS; ++i) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const Meta m0 = meta[st][i][0][u * kGroups / 4], m1 = meta[st][i][1][u * kGroups / 4];
          const uint4 w0 = dequant_unit<NBITS, OUT>(codes[st][i][0], u, m0.neg_zero, m0.scale);
          const uint4 w1 = dequant_unit<NBITS, OUT>(codes[st][i][1], u, m1.neg_zero, m1.scale);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            mma_16816<F16>(acc[i][j], w0.x, w1.x, w0.y, w1.y, x[j][4 * u], x[j][4 * u + 1]);
            mma_16816<F16>(acc[i][j], w0.z, w1.z, w0.w, w1.w, x[j][4 * u + 2], x[j][4 * u + 3]);
          }
        }
      }
      if (kb + kFewStages * kFewWarps < KB) fetch(st, kb + kFewStages * kFewWarps);
    }
  }

#pragma unroll
  for (int i = 0; i < MATS; ++i) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float* p = &red[i][warp][(8 * j + 2 * t) * kFewRedStride + g];
      p[0] = acc[i][j][0];
      p[kFewRedStride] = acc[i][j][1];
      p[8] = acc[i][j][2];
      p[kFewRedStride + 8] = acc[i][j][3];
    }
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < NT * 8 * kFewRows; idx += 32 * kFewWarps) {
    const int row = idx % kFewRows, m = idx / kFewRows;
    const int n = n0 + row, tok = tok0 + m;
    if (n >= a.N || tok >= a.M) continue;
    float v[MATS];
#pragma unroll
    for (int i = 0; i < MATS; ++i) {
      v[i] = 0.0f;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w)
        v[i] = __fadd_rn(v[i], red[i][w][m * kFewRedStride + row]);
      if (a.bias[i] != nullptr) {
        const uint32_t b = a.bias[i][n];
        v[i] = __fadd_rn(v[i], F16 ? f16_bits_to_f32(b) : bf16_bits_to_f32(b));
      }
    }
    const int64_t at = static_cast<int64_t>(tok) * a.N + n;
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
}

template <int NBITS, bool F16, int NT, int MATS>
cudaError_t launch_few_group(const FewJob& j, const FewArgs& a, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((j.N + kFewRows - 1) / kFewRows),
                  static_cast<unsigned>((j.M + 8 * NT - 1) / (8 * NT)));
  bool mm = false;
  for (int i = 0; i < MATS; ++i)
    mm = mm || a.scale_mm[i] != nullptr || a.zero_mm[i] != nullptr;
  const bool whole = j.K % 32 == 0;
  if (whole && j.group_size >= 32 && !mm)
    few_tokens_kernel<NBITS, F16, NT, MATS, 32, false><<<grid, 32 * kFewWarps, 0, st>>>(a);
  else if (whole && j.group_size >= 32)
    few_tokens_kernel<NBITS, F16, NT, MATS, 32, true><<<grid, 32 * kFewWarps, 0, st>>>(a);
  else if (whole && j.group_size == 16 && !mm)
    few_tokens_kernel<NBITS, F16, NT, MATS, 16, false><<<grid, 32 * kFewWarps, 0, st>>>(a);
  else
    few_tokens_kernel<NBITS, F16, NT, MATS, 8, true><<<grid, 32 * kFewWarps, 0, st>>>(a);
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
  a.act = j.act;
  const bool f16 = j.x_dtype == kF16, wide = j.M > 8;
  if (j.mats == 1) {
    if (f16)
      return wide ? launch_few_group<NBITS, true, 2, 1>(j, a, st)
                  : launch_few_group<NBITS, true, 1, 1>(j, a, st);
    return wide ? launch_few_group<NBITS, false, 2, 1>(j, a, st)
                : launch_few_group<NBITS, false, 1, 1>(j, a, st);
  }
  if (f16)
    return wide ? launch_few_group<NBITS, true, 2, 2>(j, a, st)
                : launch_few_group<NBITS, true, 1, 2>(j, a, st);
  return wide ? launch_few_group<NBITS, false, 2, 2>(j, a, st)
              : launch_few_group<NBITS, false, 1, 2>(j, a, st);
}

}  // namespace hqqk
