// hqq_columns.cu - W' of a weight whose groups run down its columns (axis 0), for the products on
// dequantized weights: long groups and 3-bit codes.
//
// The codes of a row block of G rows lie column by column, G of a column side by side; W' is wanted
// row by row. A block takes 128 columns of one row block, one contiguous piece of the code stream: it
// comes in by 16-byte loads, waits in shared memory (columns padded to an odd number of words) and
// goes out with a warp writing 64 neighbouring columns, 128 bytes, of a row at a time. Bound: the
// instructions of a code (issue slots 72 % taken), then HBM, 2 bytes written and nbits / 8 read per
// code. Measured, 4096 x 11008, against the kernel that writes one code per lane: 4 bits, group 64, 27 us
// (4.2 TB/s of the 6.5 a copy reaches) against 218; 2 bits, group 256, 20 against 215; 8 bits, group 64, 30
// against 227, group 16, whose blocks have 16 rows only, 58 against 215; 3 bits, 4096 x 4096, 18 against 68.
// Four columns a thread were slower (32 us at 4 bits): shared memory reads then conflict. The
// arithmetic and its three roundings are the dequantizer's.
#include "hqq_device.cuh"
#include "hqq_kernels.h"

namespace hqqk {
namespace {

constexpr int kColumns = 128, kThreads = 256;

struct ColumnArgs {
  const uint8_t* packed;
  const void *scale, *zero;
  const float *scale_mm, *zero_mm;
  int meta_run, meta_dt, group;
  int64_t cols;
  int blocks;  // of 128 columns in a row block
  uint32_t* out;
};

__device__ __forceinline__ float column_meta(const void* v, const float* mm, int dt, int run,
                                             int64_t g) {
  if (mm == nullptr) return load_meta(v, dt, g);
  const float2 p = __ldg(reinterpret_cast<const float2*>(mm) + g / run);
  return __fmul_rn(__fsub_rn(static_cast<float>(__ldg(static_cast<const uint8_t*>(v) + g)), p.y), p.x);
}

// Words of shared memory a block's codes take.
template <int NB>
__host__ __device__ constexpr int column_words(int group) {
  return NB == 3 ? (kColumns * group + 18) / 10 + 1 : kColumns * (group * NB / 32 + 1);
}

template <int NB, int OUT>
__global__ void __launch_bounds__(kThreads) columns_kernel(const ColumnArgs a) {
  extern __shared__ uint32_t words[];
  const int64_t rb = blockIdx.x / a.blocks;
  const int c0 = static_cast<int>(blockIdx.x - rb * a.blocks) * kColumns;
  const int n = static_cast<int>(a.cols - c0 < kColumns ? a.cols - c0 : kColumns);  // a multiple of 8
  const int64_t g0 = rb * a.cols + c0, e0 = g0 * a.group;
  const int per = a.group * NB / 32;  // words of a column, a multiple of 4 (not used at 3 bits)
  int slot0 = 0;
  if constexpr (NB == 3) {
    slot0 = static_cast<int>(e0 % 10);
    const uint32_t* src = reinterpret_cast<const uint32_t*>(a.packed) + e0 / 10;
    const int last = (slot0 + n * a.group - 1) / 10;
    for (int i = threadIdx.x; i <= last; i += kThreads) words[i] = __ldg(src + i);
  } else {
    const uint4* src = reinterpret_cast<const uint4*>(a.packed + e0 / 8 * NB);
    for (int i = threadIdx.x; i < n * per / 4; i += kThreads) {
      const uint4 v = __ldg(src + i);
      const int c = 4 * i / per;
      uint32_t* to = words + 4 * i + c;  // a pad word after each column
      to[0] = v.x;
      to[1] = v.y;
      to[2] = v.z;
      to[3] = v.w;
    }
  }
  __syncthreads();
  const int c = 2 * (threadIdx.x & 63), part = threadIdx.x >> 6;
  if (c >= n) return;
  float2 scale, neg_zero;
  scale.x = column_meta(a.scale, a.scale_mm, a.meta_dt, a.meta_run, g0 + c);
  scale.y = column_meta(a.scale, a.scale_mm, a.meta_dt, a.meta_run, g0 + c + 1);
  neg_zero.x = -column_meta(a.zero, a.zero_mm, a.meta_dt, a.meta_run, g0 + c);
  neg_zero.y = -column_meta(a.zero, a.zero_mm, a.meta_dt, a.meta_run, g0 + c + 1);
  const int64_t stride = a.cols / 2;  // of a row, in pairs
  uint32_t* out = a.out + rb * a.group * stride + (c0 + c) / 2;
  auto store = [&](int row, uint32_t q0, uint32_t q1) {
    const float2 neg_magic = make_float2(-8388608.0f, -8388608.0f);
    const float2 m =
        make_float2(__uint_as_float(q0 | 0x4B000000u), __uint_as_float(q1 | 0x4B000000u));
    const float2 v = fmul2_rn(fadd2_rn(fadd2_rn(m, neg_magic), neg_zero), scale);
    out[row * stride] = pack2_16<OUT>(v.x, v.y);
  };
  if constexpr (NB == 3) {
    auto code = [&](int i) {
      const uint32_t k = static_cast<uint32_t>(slot0 + i), w = k / 10u;
      return words[w] >> (3u * (k - 10u * w)) & 7u;
    };
    for (int j = part; j < a.group; j += 4)
      store(j, code(c * a.group + j), code((c + 1) * a.group + j));
  } else {
    constexpr int kCodes = 32 / NB;
    constexpr uint32_t kMask = (1u << NB) - 1u;
    const uint32_t* w0 = words + c * (per + 1);
    for (int i = part; i < per; i += 4) {
      const uint32_t x = w0[i], y = w0[i + per + 1];
#pragma unroll
      for (int b = 0; b < kCodes; ++b)
        store(i * kCodes + b, x >> (NB * b) & kMask, y >> (NB * b) & kMask);
    }
  }
}

template <int NB, int OUT>
cudaError_t launch(const DequantJob& j, cudaStream_t st) {
  ColumnArgs a;
  a.packed = j.packed;
  a.scale = j.scale;
  a.zero = j.zero;
  a.scale_mm = j.scale_mm;
  a.zero_mm = j.zero_mm;
  a.meta_run = j.meta_group_size;
  a.meta_dt = j.meta_dtype;
  a.group = j.group_size;
  a.cols = j.cols;
  a.blocks = static_cast<int>((j.cols + kColumns - 1) / kColumns);
  a.out = static_cast<uint32_t*>(j.out);
  const int64_t grid = a.blocks * (j.rows / j.group_size);
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  columns_kernel<NB, OUT>
      <<<static_cast<unsigned>(grid), kThreads, 4 * column_words<NB>(j.group_size), st>>>(a);
  return cudaGetLastError();
}

template <int NB>
cudaError_t launch_out(const DequantJob& j, cudaStream_t st) {
  return j.out_dtype == kF16 ? launch<NB, kF16>(j, st) : launch<NB, kBF16>(j, st);
}

}  // namespace

bool columns_serve(const DequantJob& j) {
  return j.axis == 0 && (j.nbits == 3 || j.nbits * j.group_size >= 128);
}

cudaError_t launch_columns(const DequantJob& j, cudaStream_t st) {
  switch (j.nbits) {
    case 1: return launch_out<1>(j, st);
    case 2: return launch_out<2>(j, st);
    case 3: return launch_out<3>(j, st);
    case 4: return launch_out<4>(j, st);
    default: return launch_out<8>(j, st);
  }
}

}  // namespace hqqk
