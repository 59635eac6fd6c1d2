// hqq_mid_2.cu - the products of some tokens at 2 bits (a translation unit of its own: they compile in
// parallel).
#include "hqq_mid_impl.cuh"

namespace hqqk {
template cudaError_t launch_mid_bits<2>(const MidJob& j, const MidPlan& plan, cudaStream_t st);
template cudaError_t read_mid_timeouts_bits<2>(unsigned int* out);
}  // namespace hqqk
