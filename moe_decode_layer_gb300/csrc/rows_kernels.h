// Host-side launchers of the many-row operators' small kernels.
#pragma once
#include <cuda_runtime.h>

#include "../../include/moe_decode_rows.h"
#include "rows_params.h"

namespace moe {
namespace rows {

// Brings the pairs (row, group) of each group together.
struct PlanParams {
  const int* idx;    // [pairs] group of each pair; outside 0..groups-1: none
  int pairs;
  int per_row;       // pairs of one row
  int groups;
  int shared;        // groups that every row belongs to, after the others
  int rows;
  int nmax;          // rows of a tile
  int keep_none;     // 1: pairs without a group get the positions after all groups'
  int align;         // groups start at multiples of it (a power of two)
  int* off;          // [groups + 1] first position of each group; keep_none: [groups + 2] and the end
  int* src_row;      // [pairs] row at each position, -1 between groups
  int* pos;          // [pairs] position of each pair or -1 (may be NULL)
  int4* ents;        // tiles (pack_tile)
  int* nent;
};
cudaError_t launch_plan(const PlanParams& p, cudaStream_t s);

// dst[p] = x[src_row[p]] for the positions p < *count that have a row
cudaError_t launch_spread(const __nv_bfloat16* x, int64_t x_stride, const int* src_row, const int* count,
                          int64_t positions, int inner, __nv_bfloat16* dst, cudaStream_t s);

// out = bf16(residual + sum_j w_j y[pos_j] + sum_s y[pairs + s * rows + row])
// residual: bf16 or (residual_f32) fp32
cudaError_t launch_combine(const float* y, const int* pos, const float* w, const void* residual, bool residual_f32,
                           __nv_bfloat16* out, int rows, int hidden, int top_k, int shared, cudaStream_t s);

// u[t, j] = scale_a sum_k A_a[j, k] x[t, k] in fp32, a = ids[t]; nothing for rows without an adapter
cudaError_t launch_shrink(const __nv_bfloat16* x, int64_t x_stride, const __nv_bfloat16* a, const float* scale,
                          const int* ids, float* u, int rows, int inner, int rank, int adapters, cudaStream_t s);

cudaError_t launch_route(const moe_route_config& c, const void* logits, int64_t stride, const float* bias,
                         int64_t rows, int32_t* idx, float* w, cudaStream_t s);

}  // namespace rows
}  // namespace moe
