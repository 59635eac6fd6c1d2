// hqq_few_3.cu - the few-token products at 3 bits (a translation unit of its own: they compile in
// parallel).
#include "hqq_few_impl.cuh"

namespace hqqk {
template cudaError_t launch_few_bits<3>(const FewJob& j, cudaStream_t st);
}  // namespace hqqk
