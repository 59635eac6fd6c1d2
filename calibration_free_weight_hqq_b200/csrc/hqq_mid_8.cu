// hqq_mid_8.cu - the products of some tokens at 8 bits (a translation unit of its own: they compile in
// parallel).
#include "hqq_mid_impl.cuh"

namespace hqqk {
template cudaError_t launch_mid_bits<8>(const MidJob& j, const MidPlan& plan, cudaStream_t st);
template cudaError_t read_mid_timeouts_bits<8>(unsigned int* out);
}  // namespace hqqk
