// hqq_few_1.cu - the few-token products at 1 bit (a translation unit of its own: they compile in
// parallel).
#include "hqq_few_impl.cuh"

namespace hqqk {
template cudaError_t launch_few_bits<1>(const FewJob& j, cudaStream_t st);
}  // namespace hqqk
