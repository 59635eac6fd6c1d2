// hqq_few_4.cu - the few-token products at 4 bits (a translation unit of its own: they compile in
// parallel).
#include "hqq_few_impl.cuh"

namespace hqqk {
template cudaError_t launch_few_bits<4>(const FewJob& j, cudaStream_t st);
}  // namespace hqqk
