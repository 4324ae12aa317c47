// Instantiations of the dense pair product for int8 weights.
#include "dense_gemm.cuh"

namespace moe {
namespace dense {

const void* pair_kernel_int8(int epi) {
  switch (epi) {
    case PAIR_SWIGLU: return reinterpret_cast<const void*>(&pair_gemm_kernel<FORM_KK8, PAIR_SWIGLU>);
    case PAIR_SWIGLU_F32: return reinterpret_cast<const void*>(&pair_gemm_kernel<FORM_KK8, PAIR_SWIGLU_F32>);
    case PAIR_F32: return reinterpret_cast<const void*>(&pair_gemm_kernel<FORM_KK8, PAIR_F32>);
    default: return reinterpret_cast<const void*>(&pair_gemm_kernel<FORM_KK8, PAIR_BF16>);
  }
}

}  // namespace dense
}  // namespace moe
