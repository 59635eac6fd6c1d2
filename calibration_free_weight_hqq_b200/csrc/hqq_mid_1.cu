// hqq_mid_1.cu - the products of some tokens at 1 bit (a translation unit of its own: they compile in
// parallel).
#include "hqq_mid_impl.cuh"

namespace hqqk {
template cudaError_t launch_mid_bits<1>(const MidJob& j, const MidPlan& plan, cudaStream_t st);
template cudaError_t read_mid_timeouts_bits<1>(unsigned int* out);
}  // namespace hqqk
