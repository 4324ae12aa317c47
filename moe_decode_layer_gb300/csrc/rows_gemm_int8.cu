// int8 instantiations of the grouped product.
#include "rows_gemm.cuh"

namespace moe {
namespace rows {

const void* gemm_kernel_int8(int epi) {
  switch (epi) {
    case EPI_SWIGLU: return reinterpret_cast<const void*>(&rows_gemm_kernel<EPI_SWIGLU, FMT_INT8>);
    case EPI_SWIGLU_F32: return reinterpret_cast<const void*>(&rows_gemm_kernel<EPI_SWIGLU_F32, FMT_INT8>);
    case EPI_F32: return reinterpret_cast<const void*>(&rows_gemm_kernel<EPI_F32, FMT_INT8>);
    default: return reinterpret_cast<const void*>(&rows_gemm_kernel<EPI_BF16, FMT_INT8>);
  }
}

}  // namespace rows
}  // namespace moe
