// FP8 instantiations of the grouped product.
#include "rows_gemm.cuh"

namespace moe {
namespace rows {

const void* gemm_kernel_fp8(int epi) {
  switch (epi) {
    case EPI_SWIGLU: return reinterpret_cast<const void*>(&rows_gemm_kernel<EPI_SWIGLU, FMT_FP8>);
    case EPI_F32: return reinterpret_cast<const void*>(&rows_gemm_kernel<EPI_F32, FMT_FP8>);
    default: return reinterpret_cast<const void*>(&rows_gemm_kernel<EPI_BF16, FMT_FP8>);
  }
}

}  // namespace rows
}  // namespace moe
