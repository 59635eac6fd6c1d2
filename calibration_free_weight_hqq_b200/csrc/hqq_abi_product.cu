// hqq_abi_product.cu - extern "C" entry points of the products over quantized weights (linear
// layers of every format, the gated pair, their gradients): argument validation, the choice of
// kernel, and the order of the launches. The contract is in include/hqq/hqq.h.
#include <algorithm>
#include <initializer_list>

#include "../../include/hqq/hqq.h"
#include "hqq_abi_internal.h"
#include "hqq_kernels.h"
#include "hqq_mid.h"

#define HQQ_EXPORT extern "C" __attribute__((visibility("default")))

static_assert((int)HQQ_ACT_SILU == hqqk::kSilu && (int)HQQ_ACT_GELU == hqqk::kGelu &&
                  (int)HQQ_ACT_GELU_TANH == hqqk::kGeluTanh,
              "activation enumerators must match");

using hqqabi::aligned;
using hqqabi::check_device;
using hqqabi::cuda_status;

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 31;

size_t weight_bytes(const hqq_weight& w) {  // the dequantized weight, 256-byte aligned
  return (static_cast<size_t>(w.rows) * static_cast<size_t>(w.cols) * 2 + 255) / 256 * 256;
}

// Everything about a weight that needs no token count: configuration, shape, pointers.
hqq_status check_weight(const hqq_weight* w) {
  if (!w) return HQQ_ERR_INVALID_ARG;
  const hqq_params& p = w->params;
  hqq_status st = hqqabi::check_shape(w->rows, w->cols, p.nbits, p.group_size, p.axis);
  if (st != HQQ_OK) return st;
  const bool qs = p.quant_scale != 0, qz = p.quant_zero != 0;
  if (!hqqabi::float_dtype(p.meta_dtype)) return HQQ_ERR_UNSUPPORTED;
  if ((qs || qz) && (st = hqqabi::check_meta_group(p.meta_group_size)) != HQQ_OK) return st;
  if ((p.flags & ~(HQQ_FLAG_STOP_AT_FIXED_POINT | HQQ_FLAG_OVERLAP_WEIGHTS)) != 0)
    return HQQ_ERR_INVALID_ARG;
  if (w->rows % 8 != 0 || w->cols % 8 != 0 || w->rows >= kMaxDim || w->cols >= kMaxDim)
    return HQQ_ERR_SHAPE;
  if (!aligned(w->bias, 2)) return HQQ_ERR_ALIGNMENT;
  if (w->rows * w->cols == 0) return HQQ_OK;
  if (!w->Wq_packed || !w->scale || !w->zero) return HQQ_ERR_INVALID_ARG;
  if ((qs && !w->scale_mm) || (qz && !w->zero_mm)) return HQQ_ERR_INVALID_ARG;
  const size_t msz = p.meta_dtype == HQQ_F32 ? 4 : 2;
  if (!aligned(w->Wq_packed, 16) || (!qs && !aligned(w->scale, msz)) ||
      (!qz && !aligned(w->zero, msz)) || (qs && !aligned(w->scale_mm, 8)) ||
      (qz && !aligned(w->zero_mm, 8)))
    return HQQ_ERR_ALIGNMENT;
  return HQQ_OK;
}

hqq_status check_pair(const hqq_weight* gate, const hqq_weight* up) {
  hqq_status st = check_weight(gate);
  if (st != HQQ_OK || (st = check_weight(up)) != HQQ_OK) return st;
  return gate->rows == up->rows && gate->cols == up->cols ? HQQ_OK : HQQ_ERR_SHAPE;
}

hqq_status check_tokens(int64_t M, int dtype) {
  if (M < 0) return HQQ_ERR_INVALID_ARG;
  if (dtype != HQQ_BF16 && dtype != HQQ_F16) return HQQ_ERR_UNSUPPORTED;
  return M < kMaxDim ? HQQ_OK : HQQ_ERR_SHAPE;
}

bool act_ok(int act) {
  return act == HQQ_ACT_SILU || act == HQQ_ACT_GELU || act == HQQ_ACT_GELU_TANH;
}

// The formats agree in everything the few-token kernel reads.
bool same_format(const hqq_params& a, const hqq_params& b) {
  return a.nbits == b.nbits && a.group_size == b.group_size && a.axis == b.axis &&
         a.meta_dtype == b.meta_dtype && !a.quant_scale == !b.quant_scale &&
         !a.quant_zero == !b.quant_zero &&
         ((!a.quant_scale && !a.quant_zero) || a.meta_group_size == b.meta_group_size);
}

hqqk::WeightView view(const hqq_weight& w) {
  hqqk::WeightView v;
  v.packed = static_cast<const uint8_t*>(w.Wq_packed);
  v.scale = w.scale;
  v.zero = w.zero;
  v.scale_mm = w.params.quant_scale ? static_cast<const float*>(w.scale_mm) : nullptr;
  v.zero_mm = w.params.quant_zero ? static_cast<const float*>(w.zero_mm) : nullptr;
  v.bias = w.bias;
  return v;
}

hqqk::FewJob few_job(int64_t M, const hqq_weight& w, const hqq_weight* up) {
  hqqk::FewJob j = {};
  j.w[0] = view(w);
  if (up) j.w[1] = view(*up);
  j.mats = up ? 2 : 1;
  j.M = M;
  j.N = w.rows;
  j.K = w.cols;
  j.nbits = w.params.nbits;
  j.group_size = w.params.group_size;
  j.meta_dtype = w.params.meta_dtype;
  j.meta_group_size = std::max(w.params.meta_group_size, 1);
  return j;
}

// Whether a forward product runs on the few-token kernel: groups along the rows, one format,
// few tokens.
bool use_few(int64_t M, const hqq_weight& w, const hqq_weight* up) {
  return w.params.axis == 1 && (up == nullptr || same_format(w.params, up->params)) &&
         hqqk::few_serves(few_job(M, w, up));
}

hqqk::MidJob mid_job(int mode, int64_t M, const hqq_weight& w, const hqq_weight* up) {
  hqqk::MidJob j = {};
  j.mode = mode;
  j.w[0] = view(w);
  if (up) j.w[1] = view(*up);
  j.weights = up ? 2 : 1;
  j.M = M;
  j.rows = w.rows;
  j.cols = w.cols;
  j.nbits = w.params.nbits;
  j.group_size = w.params.group_size;
  j.meta_dtype = w.params.meta_dtype;
  j.meta_group_size = std::max(w.params.meta_group_size, 1);
  return j;
}

// Whether a product runs straight from the codes on the some-token kernel rather than on dequantized
// weights, and what workspace that takes. Both times in us are estimated from the sizes, in millions of
// codes, partial sums and outputs:
//   * from the codes: every token tile converts the weights again, 0.26 us for a million codes and
//     0.0007 more for each token of the tile, then the partial sums;
//   * dequantized: 0.57 us for a million codes, then waves of 256 x 256 tiles over 74 CTA pairs at
//     0.33 us for 64 of the contraction, and the partial sums of a product of few tiles.
// The constants fit 480 pairs of measured times (four products, weights of 4096 x 4096, 4096 x 11008,
// 11008 x 4096 and 1024 x 8192, 1 to 8 bits, 24 to 768 tokens, all at groups of 64 with 16-bit scale and
// zero) to 9 % and 5 %; there the route taken is on average 0.5 % slower than the better one. Other formats
// are not told apart and were not fitted: from the codes, groups of 16 and 8-bit meta take longer than
// estimated, and groups of 8 and rows that are not whole 16-byte pieces several times as long. Measured in us, 4 bits, 11008 x 4096 forward and
// 4096 x 11008 backward for the first two rows, 11008 x 4096 for the others, codes / dequantized:
//   tokens       64        256         333         512         768
//   linear       24 / 50   43 / 50     62 / 72     80 / 73   102 / 74
//   gradient     25 / 48   44 / 49     63 / 69     81 / 70   105 / 71
//   gated        44 / 106  77 / 107   134 / 124   167 / 126  214 / 147
//   its grad.    42 / 89   64 / 97     90 / 120   110 / 125  159 / 169
bool use_mid(int mode, int64_t M, const hqq_weight& w, const hqq_weight* up, size_t* need) {
  if (w.params.axis != 1) return false;
  if (up != nullptr && !same_format(w.params, up->params)) return false;
  hqqk::MidPlan plan;
  if (!hqqk::mid_plan(mid_job(mode, M, w, up), &plan)) return false;
  const bool back = mode == hqqk::kMidBackward, gated = mode == hqqk::kMidGated;
  const double pair = up ? 1.0 : 0.0;
  const double codes = 1e-6 * static_cast<double>(w.rows) * static_cast<double>(w.cols) * (1 + pair);
  const int64_t out = back ? w.cols : w.rows, inner = back ? w.rows : w.cols;
  const double sums = 1e-6 * static_cast<double>(M) * static_cast<double>(out) * (gated ? 2 : 1);
  const double held = 1e-6 * plan.ctas * 2 * plan.tok * hqqk::kMidRows * (gated ? 2 : 1);
  const double direct = 8.5 + 2.2 * pair + 1.05 * held + 2.1 * sums +
                        codes * plan.tok_tiles * (0.26 + 0.0007 * plan.tok);
  const int64_t tile_n = gated ? 128 : 256;
  const int64_t tiles = ((M + 255) / 256) * ((out + tile_n - 1) / tile_n);
  const int64_t kb = (inner + 63) / 64 * (back && up ? 2 : 1);
  const int kind = back ? hqqk::kDenseBackward : up ? hqqk::kDenseGated : hqqk::kDenseForward;
  const int parts = hqqk::dense_splits(kind, M, out, inner, up ? 2 : 1);
  const double dense = 6.4 + 3.6 * pair + 0.57 * codes + (parts > 1 ? 1.8 * parts * sums : 0.0) +
                       0.33 * static_cast<double>((tiles * parts + 73) / 74) *
                           static_cast<double>((kb + parts - 1) / parts);
  if (direct > dense) return false;
  *need = (plan.partial_bytes + 255) / 256 * 256;
  return true;
}

// The dequantized weights, then the partial sums of a product of few tiles.
size_t dense_weights(const hqq_weight& w, const hqq_weight* up) {
  return weight_bytes(w) + (up ? weight_bytes(*up) : 0);
}

size_t dense_need(int kind, int64_t M, const hqq_weight& w, const hqq_weight* up) {
  const bool back = kind == hqqk::kDenseBackward;
  return dense_weights(w, up) + hqqk::dense_partial_bytes(kind, M, back ? w.cols : w.rows,
                                                          back ? w.rows : w.cols, up ? 2 : 1);
}

size_t forward_need(int64_t M, const hqq_weight& w, const hqq_weight* up) {
  size_t need = 0;
  if (M == 0 || w.rows == 0 || w.cols == 0 || use_few(M, w, up)) return 0;
  if (use_mid(up ? hqqk::kMidGated : hqqk::kMidLinear, M, w, up, &need)) return need;
  return dense_need(up ? hqqk::kDenseGated : hqqk::kDenseForward, M, w, up);
}

size_t backward_need(int64_t M, const hqq_weight& w, const hqq_weight* up) {
  size_t need = 0;
  if (M == 0 || w.rows == 0 || w.cols == 0) return 0;
  if (use_mid(hqqk::kMidBackward, M, w, up, &need)) return need;
  return dense_need(hqqk::kDenseBackward, M, w, up);
}

hqqk::DequantJob dequant_job(const hqq_weight& w, int dtype, void* out) {
  const hqqk::WeightView v = view(w);
  hqqk::DequantJob j;
  j.packed = v.packed;
  j.scale = v.scale;
  j.zero = v.zero;
  j.scale_mm = v.scale_mm;
  j.zero_mm = v.zero_mm;
  j.meta_group_size = w.params.meta_group_size;
  j.meta_dtype = w.params.meta_dtype;
  j.rows = w.rows;
  j.cols = w.cols;
  j.n_groups = w.rows * w.cols / w.params.group_size;
  j.nbits = w.params.nbits;
  j.group_size = w.params.group_size;
  j.axis = w.params.axis;
  j.out_dtype = dtype;
  j.out = out;
  return j;
}

hqq_status dequantize_one(const hqqk::DequantJob& j, cudaStream_t stream) {
  return cuda_status(hqqk::columns_serve(j) ? hqqk::launch_columns(j, stream)
                                            : hqqk::launch_dequantize(j, stream));
}

// The weight, or both of a pair, dequantized into the workspace, one after the other: W'[i] in
// out[i].
hqq_status dequantize_into(void* workspace, const hqq_weight& w, const hqq_weight* up, int dtype,
                           const void* (&out)[2], cudaStream_t stream) {
  out[0] = workspace;
  out[1] = static_cast<char*>(workspace) + (up ? weight_bytes(w) : 0);
  const hqq_status st = dequantize_one(dequant_job(w, dtype, const_cast<void*>(out[0])), stream);
  if (st != HQQ_OK || !up) return st;
  return dequantize_one(dequant_job(*up, dtype, const_cast<void*>(out[1])), stream);
}

hqq_status check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (need == 0) return HQQ_OK;
  if (!workspace || bytes < need) return HQQ_ERR_WORKSPACE;
  return aligned(workspace, 16) ? HQQ_OK : HQQ_ERR_ALIGNMENT;
}

struct Range {
  const void* p;
  size_t bytes;
};

// HQQ_ERR_INVALID_ARG where one of the first `outputs` ranges (or the workspace, counted among them)
// overlaps another range: the kernels read while they write.
hqq_status check_apart(std::initializer_list<Range> ranges, size_t outputs) {
  const Range* const r = ranges.begin();
  for (size_t i = 0; i < outputs; ++i)
    for (size_t j = i + 1; j < ranges.size(); ++j) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(r[i].p), b = reinterpret_cast<uintptr_t>(r[j].p);
      if (a != 0 && b != 0 && r[i].bytes != 0 && r[j].bytes != 0 && a < b + r[j].bytes &&
          b < a + r[i].bytes)
        return HQQ_ERR_INVALID_ARG;
    }
  return HQQ_OK;
}

size_t token_bytes(int64_t M, int64_t width) {
  return static_cast<size_t>(M) * static_cast<size_t>(width) * 2;
}

hqq_status forward(const void* X, int64_t M, int dtype, const hqq_weight& w, const hqq_weight* up,
                   int act, void* Y, void* G, void* U, void* workspace, size_t workspace_bytes,
                   cudaStream_t stream) {
  if (M == 0 || w.rows == 0) return HQQ_OK;
  if (!Y || (w.cols > 0 && !X)) return HQQ_ERR_INVALID_ARG;
  if (!aligned(X, 16) || !aligned(Y, 16) || !aligned(G, 16) || !aligned(U, 16))
    return HQQ_ERR_ALIGNMENT;
  const size_t need = forward_need(M, w, up), out = token_bytes(M, w.rows);
  hqq_status st = check_workspace(workspace, workspace_bytes, need);
  if (st == HQQ_OK)
    st = check_apart({{Y, out}, {G, out}, {U, out}, {workspace, need}, {X, token_bytes(M, w.cols)}}, 4);
  if (st != HQQ_OK) return st;
  if ((st = check_device(w.cols > 0 ? X : Y)) != HQQ_OK) return st;
  if (w.cols == 0) {
    const void* const bias[2] = {w.bias, up ? up->bias : nullptr};
    return cuda_status(hqqk::launch_empty_sums(bias, up ? 2 : 1, M, w.rows, dtype, act, Y, G, U,
                                               stream));
  }
  if (use_few(M, w, up)) {
    hqqk::FewJob j = few_job(M, w, up);
    j.X = X;
    j.x_dtype = dtype;
    j.act = act;
    j.Y = Y;
    j.G = G;
    j.U = U;
    return cuda_status(hqqk::launch_few(j, stream));
  }
  const int mode = up ? hqqk::kMidGated : hqqk::kMidLinear;
  if (size_t need = 0; use_mid(mode, M, w, up, &need)) {
    hqqk::MidJob j = mid_job(mode, M, w, up);
    j.X[0] = X;
    j.x_dtype = dtype;
    j.act = act;
    j.Y = Y;
    j.G = G;
    j.U = U;
    j.workspace = workspace;
    return cuda_status(hqqk::launch_mid(j, stream));
  }
  hqqk::DenseJob j = {};
  if ((st = dequantize_into(workspace, w, up, dtype, j.B, stream)) != HQQ_OK) return st;
  j.kind = up ? hqqk::kDenseGated : hqqk::kDenseForward;
  j.A[0] = X;
  j.bias[0] = w.bias;
  j.bias[1] = up ? up->bias : nullptr;
  j.sources = 1;
  j.M = M;
  j.N = w.rows;
  j.K = w.cols;
  j.x_dtype = dtype;
  j.act = act;
  j.partial = static_cast<char*>(workspace) + dense_weights(w, up);
  j.D = Y;
  j.G = G;
  j.U = U;
  return cuda_status(hqqk::launch_dense(j, stream));
}

// dX[M, cols] = sum over the weights of A[i][M, rows] W'[i].
hqq_status backward(const void* const (&A)[2], int64_t M, int dtype, const hqq_weight& w,
                    const hqq_weight* up, void* dX, void* workspace, cudaStream_t stream) {
  if (M == 0 || w.cols == 0) return HQQ_OK;
  if (w.rows == 0)  // an empty sum
    return cuda_status(cudaMemsetAsync(dX, 0, static_cast<size_t>(M) * w.cols * 2, stream));
  if (size_t need = 0; use_mid(hqqk::kMidBackward, M, w, up, &need)) {
    hqqk::MidJob j = mid_job(hqqk::kMidBackward, M, w, up);
    j.X[0] = A[0];
    j.X[1] = A[1];
    j.x_dtype = dtype;
    j.Y = dX;
    j.workspace = workspace;
    return cuda_status(hqqk::launch_mid(j, stream));
  }
  hqqk::DenseJob j = {};
  const hqq_status st = dequantize_into(workspace, w, up, dtype, j.B, stream);
  if (st != HQQ_OK) return st;
  j.kind = hqqk::kDenseBackward;
  j.A[0] = A[0];
  j.A[1] = A[1];
  j.sources = up ? 2 : 1;
  j.M = M;
  j.N = w.cols;
  j.K = w.rows;
  j.x_dtype = dtype;
  j.partial = static_cast<char*>(workspace) + dense_weights(w, up);
  j.D = dX;
  return cuda_status(hqqk::launch_dense(j, stream));
}

}  // namespace

HQQ_EXPORT size_t hqq_linear_workspace_bytes(int64_t M, const hqq_weight* w, int backward_pass) {
  if (M < 0 || M >= kMaxDim || check_weight(w) != HQQ_OK) return static_cast<size_t>(-1);
  return backward_pass ? backward_need(M, *w, nullptr) : forward_need(M, *w, nullptr);
}

HQQ_EXPORT size_t hqq_gated_linear_workspace_bytes(int64_t M, const hqq_weight* gate,
                                                   const hqq_weight* up, int backward_pass) {
  if (M < 0 || M >= kMaxDim || check_pair(gate, up) != HQQ_OK) return static_cast<size_t>(-1);
  return backward_pass ? backward_need(M, *gate, up) : forward_need(M, *gate, up);
}

HQQ_EXPORT hqq_status hqq_linear_ex(const void* X, int64_t M, hqq_dtype x_dtype,
                                    const hqq_weight* w, void* Y, void* workspace,
                                    size_t workspace_bytes, cudaStream_t stream) {
  hqq_status st = check_weight(w);
  if (st != HQQ_OK || (st = check_tokens(M, x_dtype)) != HQQ_OK) return st;
  return forward(X, M, x_dtype, *w, nullptr, HQQ_ACT_SILU, Y, nullptr, nullptr, workspace,
                 workspace_bytes, stream);
}

HQQ_EXPORT hqq_status hqq_gated_linear(const void* X, int64_t M, hqq_dtype x_dtype,
                                       const hqq_weight* gate, const hqq_weight* up, hqq_act act,
                                       void* Y, void* G, void* U, void* workspace,
                                       size_t workspace_bytes, cudaStream_t stream) {
  hqq_status st = check_pair(gate, up);
  if (st != HQQ_OK || (st = check_tokens(M, x_dtype)) != HQQ_OK) return st;
  if (!act_ok(act)) return HQQ_ERR_UNSUPPORTED;
  return forward(X, M, x_dtype, *gate, up, act, Y, G, U, workspace, workspace_bytes, stream);
}

HQQ_EXPORT hqq_status hqq_linear_backward(const void* dY, int64_t M, hqq_dtype x_dtype,
                                          const hqq_weight* w, void* dX, void* dbias,
                                          void* workspace, size_t workspace_bytes,
                                          cudaStream_t stream) {
  hqq_status st = check_weight(w);
  if (st != HQQ_OK || (st = check_tokens(M, x_dtype)) != HQQ_OK) return st;
  const bool product = M > 0 && w->cols > 0, sums = dbias != nullptr && w->rows > 0;
  if (!product && !sums) return HQQ_OK;
  if ((product && !dX) || (M > 0 && w->rows > 0 && !dY)) return HQQ_ERR_INVALID_ARG;
  if (!aligned(dY, 16) || !aligned(dX, 16) || !aligned(dbias, 2)) return HQQ_ERR_ALIGNMENT;
  const size_t need = product ? backward_need(M, *w, nullptr) : 0;
  st = check_workspace(workspace, workspace_bytes, need);
  if (st == HQQ_OK)
    st = check_apart({{dX, token_bytes(M, w->cols)}, {dbias, token_bytes(1, w->rows)}, {workspace, need},
                      {dY, token_bytes(M, w->rows)}}, 3);
  if (st != HQQ_OK) return st;
  if ((st = check_device(dY ? dY : product ? dX : dbias)) != HQQ_OK) return st;
  const void* A[2] = {dY, nullptr};
  if ((st = backward(A, M, x_dtype, *w, nullptr, dX, workspace, stream)) != HQQ_OK) return st;
  if (!sums) return HQQ_OK;
  return cuda_status(
      hqqk::launch_column_sums(dY, dbias, nullptr, nullptr, M, w->rows, x_dtype, stream));
}

HQQ_EXPORT hqq_status hqq_gated_linear_backward(const void* dY, const void* G, const void* U,
                                                int64_t M, hqq_dtype x_dtype,
                                                const hqq_weight* gate, const hqq_weight* up,
                                                hqq_act act, void* dG, void* dU, void* dX,
                                                void* dbias_gate, void* dbias_up, void* workspace,
                                                size_t workspace_bytes, cudaStream_t stream) {
  hqq_status st = check_pair(gate, up);
  if (st != HQQ_OK || (st = check_tokens(M, x_dtype)) != HQQ_OK) return st;
  if (!act_ok(act)) return HQQ_ERR_UNSUPPORTED;
  const int64_t N = gate->rows, K = gate->cols;
  const bool product = M > 0 && K > 0, rows = M > 0 && N > 0;
  const bool sums = N > 0 && (dbias_gate != nullptr || dbias_up != nullptr);
  if (!product && !rows && !sums) return HQQ_OK;
  if ((rows && (!dY || !G || !U || !dG || !dU)) || (product && !dX)) return HQQ_ERR_INVALID_ARG;
  for (const void* p : {dY, G, U, static_cast<const void*>(dG), static_cast<const void*>(dU),
                        static_cast<const void*>(dX)})
    if (!aligned(p, 16)) return HQQ_ERR_ALIGNMENT;
  if (!aligned(dbias_gate, 2) || !aligned(dbias_up, 2)) return HQQ_ERR_ALIGNMENT;
  const size_t need = product ? backward_need(M, *gate, up) : 0, wide = token_bytes(M, N);
  st = check_workspace(workspace, workspace_bytes, need);
  if (st == HQQ_OK)
    st = check_apart({{dX, token_bytes(M, K)}, {dG, wide}, {dU, wide}, {dbias_gate, token_bytes(1, N)},
                      {dbias_up, token_bytes(1, N)}, {workspace, need}, {dY, wide}, {G, wide}, {U, wide}},
                     6);
  if (st != HQQ_OK) return st;
  const void* first = rows ? dY : product ? dX : dbias_gate ? dbias_gate : dbias_up;
  if ((st = check_device(first)) != HQQ_OK) return st;
  if (rows)
    st = cuda_status(hqqk::launch_gated_grad(dY, G, U, M * N, x_dtype, act, dG, dU, stream));
  if (st != HQQ_OK) return st;
  const void* A[2] = {dG, dU};
  if ((st = backward(A, M, x_dtype, *gate, up, dX, workspace, stream)) != HQQ_OK) return st;
  if (!sums) return HQQ_OK;
  return cuda_status(
      hqqk::launch_column_sums(dG, dbias_gate, dU, dbias_up, M, N, x_dtype, stream));
}
