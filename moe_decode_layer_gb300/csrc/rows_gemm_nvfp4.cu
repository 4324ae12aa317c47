// NVFP4 instantiations of the grouped product.
#include "rows_gemm.cuh"

namespace moe {
namespace rows {

const void* gemm_kernel_nvfp4(int epi) {
  switch (epi) {
    case EPI_SWIGLU: return reinterpret_cast<const void*>(&rows_gemm_kernel<EPI_SWIGLU, FMT_NVFP4>);
    case EPI_F32: return reinterpret_cast<const void*>(&rows_gemm_kernel<EPI_F32, FMT_NVFP4>);
    default: return reinterpret_cast<const void*>(&rows_gemm_kernel<EPI_BF16, FMT_NVFP4>);
  }
}

}  // namespace rows
}  // namespace moe
