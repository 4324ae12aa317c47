// Instantiations of the dense pair product for k-innermost operands, and the table of all.
#include "dense_gemm.cuh"

namespace moe {
namespace dense {

const void* pair_kernel_backward(int form, int epi);
const void* pair_kernel_int8(int epi);

const void* pair_kernel(int form, int epi) {
  if (form == FORM_KK8) return pair_kernel_int8(epi);
  if (form != FORM_KK) return pair_kernel_backward(form, epi);
  return epi == PAIR_SWIGLU ? reinterpret_cast<const void*>(&pair_gemm_kernel<FORM_KK, PAIR_SWIGLU>)
                            : reinterpret_cast<const void*>(&pair_gemm_kernel<FORM_KK, PAIR_BF16>);
}

}  // namespace dense
}  // namespace moe
