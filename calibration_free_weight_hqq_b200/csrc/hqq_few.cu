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

// A pair in groups of 16 with 8-bit or fp32 meta does not fit the registers here and is left to the
// some-token kernel (11008 x 4096, 2 bits, 8-bit meta, 1 token: 87 us here, 60 there).
bool few_serves(const FewJob& j) {
  bool wide_meta = j.meta_dtype == kF32;
  for (int i = 0; i < j.mats; ++i)
    wide_meta = wide_meta || j.w[i].scale_mm != nullptr || j.w[i].zero_mm != nullptr;
  return few_warps(j) > 0 && !(j.mats == 2 && j.group_size == 16 && wide_meta);
}

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
