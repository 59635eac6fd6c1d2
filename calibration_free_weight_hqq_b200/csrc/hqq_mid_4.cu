// hqq_mid_4.cu - the products of some tokens at 4 bits (a translation unit of its own: they compile in
// parallel).
#include "hqq_mid_impl.cuh"

namespace hqqk {
template cudaError_t launch_mid_bits<4>(const MidJob& j, const MidPlan& plan, cudaStream_t st);
template cudaError_t read_mid_timeouts_bits<4>(unsigned int* out);
}  // namespace hqqk
