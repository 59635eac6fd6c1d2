// hqq_few_8.cu - the few-token products at 8 bits (a translation unit of its own: they compile in
// parallel).
#include "hqq_few_impl.cuh"

namespace hqqk {
template cudaError_t launch_few_bits<8>(const FewJob& j, cudaStream_t st);
}  // namespace hqqk
