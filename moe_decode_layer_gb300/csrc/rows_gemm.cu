// Instantiations of the grouped product for bf16 weights and the table of all.
#include "rows_gemm.cuh"

namespace moe {
namespace rows {

const void* gemm_kernel_fp8(int epi);
const void* gemm_kernel_nvfp4(int epi);

const void* gemm_kernel(int epi, int fmt) {
  if (fmt == FMT_FP8) return gemm_kernel_fp8(epi);
  if (fmt == FMT_NVFP4) return gemm_kernel_nvfp4(epi);
  switch (epi) {
    case EPI_SWIGLU: return reinterpret_cast<const void*>(&rows_gemm_kernel<EPI_SWIGLU, FMT_BF16>);
    case EPI_F32: return reinterpret_cast<const void*>(&rows_gemm_kernel<EPI_F32, FMT_BF16>);
    case EPI_TWO: return reinterpret_cast<const void*>(&rows_gemm_kernel<EPI_TWO, FMT_BF16>);
    default: return reinterpret_cast<const void*>(&rows_gemm_kernel<EPI_BF16, FMT_BF16>);
  }
}

}  // namespace rows
}  // namespace moe
