// Instantiations of the dense pair product for the backward pass.
#include "dense_gemm.cuh"

namespace moe {
namespace dense {

const void* pair_kernel_backward(int form, int epi) {
  if (form == FORM_KM)
    return epi == PAIR_DSWIGLU      ? reinterpret_cast<const void*>(&pair_gemm_kernel<FORM_KM, PAIR_DSWIGLU>)
           : epi == PAIR_DSWIGLU_LO ? reinterpret_cast<const void*>(&pair_gemm_kernel<FORM_KM, PAIR_DSWIGLU_LO>)
                                    : reinterpret_cast<const void*>(&pair_gemm_kernel<FORM_KM, PAIR_BF16>);
  return epi == PAIR_F32 ? reinterpret_cast<const void*>(&pair_gemm_kernel<FORM_MM, PAIR_F32>)
                         : reinterpret_cast<const void*>(&pair_gemm_kernel<FORM_MM, PAIR_BF16>);
}

}  // namespace dense
}  // namespace moe
