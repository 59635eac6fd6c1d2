// hqq_few.cu - picks the few-token product's instantiation by code width (hqq_few_impl.cuh).
#include "hqq_few.h"
#include "hqq_kernels.h"

namespace hqqk {

template <int NBITS>
cudaError_t launch_few_bits(const FewJob& j, cudaStream_t st);
extern template cudaError_t launch_few_bits<1>(const FewJob&, cudaStream_t);
extern template cudaError_t launch_few_bits<2>(const FewJob&, cudaStream_t);
extern template cudaError_t launch_few_bits<3>(const FewJob&, cudaStream_t);
extern template cudaError_t launch_few_bits<4>(const FewJob&, cudaStream_t);
extern template cudaError_t launch_few_bits<8>(const FewJob&, cudaStream_t);

bool few_serves(const FewJob& j) { return few_warps(j) > 0; }

cudaError_t launch_few(const FewJob& j, cudaStream_t st) {
  switch (j.nbits) {
    case 1: return launch_few_bits<1>(j, st);
    case 2: return launch_few_bits<2>(j, st);
    case 3: return launch_few_bits<3>(j, st);
    case 4: return launch_few_bits<4>(j, st);
    default: return launch_few_bits<8>(j, st);
  }
}

}  // namespace hqqk
