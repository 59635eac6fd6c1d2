// hqq_kernels.h - host-side launch interface between the C ABI layer and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace hqqk {

// Element types; the values equal the public hqq_dtype enumerators.
enum Dt : int { kF16 = 0, kBF16 = 1, kF32 = 2, kU8 = 3 };

// One matrix of the quantize path.
struct QuantJob {
  const void* W;     // device, row-major [rows, cols]
  int64_t rows, cols, n_groups;
  int w_dtype;       // Dt
  int nbits, group_size, axis, iters;
  float p, beta0, kappa;
  uint8_t* packed;   // device, packed code stream
  void* scale;       // device, n_groups values of scale_dtype
  void* zero;        // device, n_groups values of zero_dtype
  int scale_dtype;   // Dt (kF32 when the second level follows)
  int zero_dtype;
  int flags;         // HQQ_FLAG_* bits
};

// One matrix of the dequantize path.
struct DequantJob {
  const uint8_t* packed;
  const void* scale;  // meta_dtype values, or uint8 codes when scale_mm != nullptr
  const void* zero;   // meta_dtype values, or uint8 codes when zero_mm != nullptr
  const float* scale_mm;  // second-level (step2, zero2) pairs or nullptr
  const float* zero_mm;
  int meta_group_size;
  int meta_dtype;
  int64_t rows, cols, n_groups;
  int nbits, group_size, axis;
  int out_dtype;
  void* out;
};

// Matrices per batched launch (their pointers and tile prefix sums travel as kernel
// parameters); larger batches are split into several launches.
constexpr int kMaxBatch = 256;

cudaError_t launch_quantize(const QuantJob& job, cudaStream_t stream);
// All jobs share nbits, group_size, axis, iters, p, beta0, kappa and the dtypes.
cudaError_t launch_quantize_batched(const QuantJob* jobs, int n, cudaStream_t stream);
cudaError_t launch_dequantize(const DequantJob& job, cudaStream_t stream);
// All jobs share the settings and dtypes; only pointers and shapes differ.
cudaError_t launch_dequantize_batched(const DequantJob* jobs, int n, cudaStream_t stream);
// Y[M, N] = X[M, K] · W'^T (+ bias) with W' the dequantized 4-bit, group-64, axis-1 weight
// [N, K]; X, bias and Y share x_dtype (kBF16 or kF16). Shapes and alignment are validated by
// the caller: K % 64 == 0, N % 8 == 0, 16-byte aligned X, packed and Y.
struct GemmJob {
  const void* X;
  const uint8_t* packed;
  const void* scale;
  const void* zero;
  const void* bias;  // nullptr or [N]
  void* Y;
  int64_t M, N, K;
  int x_dtype;
  int meta_dtype;
  bool overlap_weights;  // HQQ_FLAG_OVERLAP_WEIGHTS: the decode kernel may overlap the
                         // previous kernel on the stream (programmatic dependent launch)
};
cudaError_t launch_w4a16_gemm(const GemmJob& job, cudaStream_t stream);
// Number of bounded waits inside the GEMM kernel that ran out of time since the library was
// loaded (0 on every healthy run).
cudaError_t read_gemm_timeouts(unsigned int* out);

// Activations of the gated products; the values equal the public hqq_act enumerators.
enum Act : int { kSilu = 0, kGelu = 1, kGeluTanh = 2 };

// A quantized weight [N, K] of a product; bias: nullptr or [N] of the activation dtype.
struct WeightView {
  const uint8_t* packed;
  const void* scale;  // meta_dtype values, or uint8 codes when scale_mm != nullptr
  const void* zero;
  const float* scale_mm;
  const float* zero_mm;
  const void* bias;
};

// Product of up to 8 tokens with one weight (mats = 1: Y = X W'^T + bias) or the gated pair (mats = 2:
// Y = act(X Wg'^T + bg) * (X Wu'^T + bu)); axis 1, any nbits and group size, both weights of
// one format. G, U: nullptr or where the gated pair's projections go, rounded.
struct FewJob {
  const void* X;
  WeightView w[2];
  int mats;
  int64_t M, N, K;
  int x_dtype;
  int nbits, group_size, meta_dtype, meta_group_size;
  int act;
  void *Y, *G, *U;
};
// Whether launch_few takes a job of these sizes and format (up to 8 tokens whose X fits).
bool few_serves(const FewJob& job);
cudaError_t launch_few(const FewJob& job, cudaStream_t stream);

// Large products on dequantized weights (x_dtype, row-major), on the 2-SM tensor-core kernel.
enum DenseKind : int {
  kDenseForward = 0,   // D[M, N] = A[0][M, K] B[0][N, K]^T (+ bias[0])
  kDenseGated = 1,     // D[M, N] = act(A[0] B[0]^T + bias[0]) * (A[0] B[1]^T + bias[1]); G, U
  kDenseBackward = 2,  // D[M, N] = sum over i < sources of A[i][M, K] B[i][K, N]
};
struct DenseJob {
  int kind;
  const void* A[2];
  const void* B[2];
  const void* bias[2];
  int sources;  // of kDenseBackward: 1 or 2
  int64_t M, N, K;
  int x_dtype;
  int act;
  void *D, *G, *U;
  void* partial;  // dense_partial_bytes of workspace
};
// Parts of the contraction a product is cut into, and the workspace their sums take (0 for one part).
int dense_splits(int kind, int64_t M, int64_t N, int64_t K, int sources);
size_t dense_partial_bytes(int kind, int64_t M, int64_t N, int64_t K, int sources);
cudaError_t launch_dense(const DenseJob& job, cudaStream_t stream);
cudaError_t read_dense_timeouts(unsigned int* out);

// Dequantization of an axis-0 weight of 8 | cols to 16 bits, for long groups and 3-bit codes
// (columns_serve); values as launch_dequantize writes them.
bool columns_serve(const DequantJob& job);
cudaError_t launch_columns(const DequantJob& job, cudaStream_t stream);

// Products over weights of no columns: every sum is its bias (or 0).
cudaError_t launch_empty_sums(const void* const (&bias)[2], int mats, int64_t M, int64_t N,
                              int x_dtype, int act, void* Y, void* G, void* U,
                              cudaStream_t stream);

// dG = dY * U * act'(G), dU = dY * act(G), elementwise over n values of x_dtype.
cudaError_t launch_gated_grad(const void* dY, const void* G, const void* U, int64_t n, int x_dtype,
                              int act, void* dG, void* dU, cudaStream_t stream);
// out0[c] = sum over rows of A0[rows, cols] and out1 of A1, fp32 in a fixed order, rounded once; those
// without an out are left.
cudaError_t launch_column_sums(const void* A0, void* out0, const void* A1, void* out1, int64_t rows,
                               int64_t cols, int x_dtype, cudaStream_t stream);

// MXFP4: n = rows*cols elements (n % 32 == 0), blocks of 32 consecutive elements.
cudaError_t launch_mxfp4_quantize(const void* W, int dtype, int64_t n, uint8_t* codes,
                                  uint8_t* scales, cudaStream_t stream);
cudaError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t n,
                                    int out_dtype, void* out, cudaStream_t stream);

cudaError_t launch_quantize_meta(const void* meta, int dtype, int64_t n, int group, uint8_t* q,
                                 float* mm, cudaStream_t stream);
cudaError_t launch_dequantize_meta(const uint8_t* q, const float* mm, int64_t n, int group,
                                   float* out, cudaStream_t stream);

}  // namespace hqqk
