// hqq_mid.cu - the division of work of the products of some tokens (hqq_mid_impl.cuh) and the choice of
// their instantiation by code width.
#include "hqq_mid.h"

#include <algorithm>

namespace hqqk {

template <int NBITS>
cudaError_t launch_mid_bits(const MidJob& j, const MidPlan& plan, cudaStream_t st);
template <int NBITS>
cudaError_t read_mid_timeouts_bits(unsigned int* out);

bool mid_plan(const MidJob& j, MidPlan* plan) {
  const bool back = j.mode == kMidBackward;
  const int64_t out = back ? j.cols : j.rows, inner = back ? j.rows : j.cols;
  if (j.M < 1 || out < 1 || inner < 1 || j.cols > kMidMaxCols) return false;
  MidPlan p = {};
  const int64_t tok_tiles = (j.M + kMidTokens - 1) / kMidTokens;
  p.tok = static_cast<int>(((j.M + tok_tiles - 1) / tok_tiles + 15) / 16 * 16);
  const int64_t row_tiles = (out + kMidRows - 1) / kMidRows;
  p.kb1 = static_cast<int>((inner + mid_bk(j.mode) - 1) / mid_bk(j.mode));
  p.kb = back ? p.kb1 * j.weights : p.kb1;
  const int64_t units = row_tiles * tok_tiles * p.kb;
  if (units > 0x3FFFFFFF) return false;
  p.tok_tiles = static_cast<int>(tok_tiles);
  p.row_tiles = static_cast<int>(row_tiles);
  // every SM, but at least two k-blocks each: fewer cost more in partial tiles than they save
  p.ctas = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kSms, units / 2)));
  const uint32_t ring = static_cast<uint32_t>(kMidDqWarps * mid_codes(j.nbits, j.mode) * mid_depth(j.nbits, j.mode));
  const uint32_t stage = 2 * kMidTileBytes + static_cast<uint32_t>(p.tok) * 2 * mid_bk(j.mode);
  p.stages = static_cast<int>(std::min<uint32_t>(4, (kMidMaxSmem - 2048u - ring) / stage));
  p.off_ring = p.stages * stage;
  p.off_bar = p.off_ring + ring;
  p.smem = p.off_bar + 1024 + 1024;  // barriers, TMEM address and flag; slack to align the base
  p.partial_bytes = static_cast<size_t>(p.ctas) * 2 * (j.mode == kMidGated ? 2 : 1) * p.tok *
                    kMidRows * sizeof(float);
  *plan = p;
  return true;
}

cudaError_t launch_mid(const MidJob& j, cudaStream_t st) {
  MidPlan plan;
  if (!mid_plan(j, &plan)) return cudaErrorInvalidValue;
  switch (j.nbits) {
    case 1: return launch_mid_bits<1>(j, plan, st);
    case 2: return launch_mid_bits<2>(j, plan, st);
    case 3: return launch_mid_bits<3>(j, plan, st);
    case 4: return launch_mid_bits<4>(j, plan, st);
    default: return launch_mid_bits<8>(j, plan, st);
  }
}

cudaError_t read_mid_timeouts(unsigned int* out) {
  unsigned int n[5] = {};
  cudaError_t e = read_mid_timeouts_bits<1>(&n[0]);
  if (e == cudaSuccess) e = read_mid_timeouts_bits<2>(&n[1]);
  if (e == cudaSuccess) e = read_mid_timeouts_bits<3>(&n[2]);
  if (e == cudaSuccess) e = read_mid_timeouts_bits<4>(&n[3]);
  if (e == cudaSuccess) e = read_mid_timeouts_bits<8>(&n[4]);
  if (e == cudaSuccess) *out = n[0] + n[1] + n[2] + n[3] + n[4];
  return e;
}

}  // namespace hqqk
