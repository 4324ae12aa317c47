// Launch parameters of the dense operators' kernels, shared by the host code
// (dense_api.cu) and the kernels.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "rows_params.h"

namespace moe {
namespace dense {

constexpr int kPairStages = 16;      // operand stages at most
constexpr int kTileM = 256;          // rows of a pair's tile
constexpr int kRawSlots = 6;         // slots of codes at most
constexpr int kStageBox = 4096;      // an epilogue warp's box in shared memory: 32 rows of 128 bytes
constexpr int kSplitMost = 4;        // pairs of a cluster of 8
constexpr int kGroupM = 8;           // row tiles that go round the columns together

// Which of the operands lies with its own index innermost (MN-major), not with k's.
enum Form {
  FORM_KK = 0,  // A [M, K], B [N, K]
  FORM_KM = 1,  // A [M, K], B [K, N]
  FORM_MM = 2,  // A [K, M], B [K, N]
  FORM_KK8 = 3  // FORM_KK, fp16 A and int8 B, which is widened to fp16 in shared memory
};
// Copies, tensor core, copies of codes, an idle warp; eight epilogue warps, or (FORM_KK8) four and eight that widen.
__host__ __device__ constexpr int pair_threads(int form) { return form == FORM_KK8 ? 512 : 384; }
enum PairEpi {
  PAIR_BF16 = 0,
  PAIR_F32 = 1,
  PAIR_SWIGLU = 2,      // bf16 silu(gate) * up, and (map_e) gate and up themselves
  PAIR_SWIGLU_F32 = 3,  // the same in fp32, without them
  PAIR_DSWIGLU = 4,     // from dh, gate and up: bf16 dg, du (map_e) and h
  PAIR_DSWIGLU_LO = 5   // each as two bf16 numbers, the second ones in the maps' later halves
};

struct PairParams {
  int M, N, K;   // SWIGLU: N columns of h, 2 N rows of B
  int bn;        // accumulator columns of a tile, 256, 192 or 128 (SWIGLU: half gate, half up; not 192)
  int tiles_m, tiles_n;
  int M2, N2, tiles_m2, tiles_n2;  // FORM_MM: a second product over the same K, behind the first's tiles (tiles_m2 0: none)
  int split;     // pairs of a cluster that share a tile's K
  int stages, stage_bytes;
  int raw_off, raw_slots;  // FORM_KK8: slots of 128 codes of each row of B
  // A's part of a stage: 128 rows, or of few rows (M <= 128, no FORM_MM) those in the first CTA alone.
  // The tensor core reads 128 all the same; what lies behind them becomes rows that nothing reads.
  int a_bytes;
  int step_bytes;  // both CTAs' copies of a step
  int ewarps;    // epilogue warps at work, 8 or 4
  int bufs;      // boxes of an epilogue warp
  int box_off;   // where they are: behind the stages, and behind a split tile's sums
  int ahead;     // steps of B that are fetched to L2 before their copies, or 0
  uint32_t idesc;
  const float* row_scale;  // FORM_KK8: a scale for each row and each column (gate columns first)
  const float* col_scale;
  int scale_off;           // the scales of a tile's columns, for each epilogue warp
  const __nv_bfloat16* addend;  // [M, N], or NULL
  // An operand that is the sum of two bf16 numbers: K is gone through twice (passes 2), the second time this many
  // columns further on in A and in B (and in the second product's).
  int passes, pass_a, pass_b, pass_a2, pass_b2;
  int keep;      // SWIGLU: store gate and up; DSWIGLU, DSWIGLU_LO: store h
  int reduce;    // F32: add to what is there
  int pdl;
  int* status;   // one word a CTA; 1 = a wait ran into its limit
  int status_keep;  // 1: not the call's first launch with waits; words are only set
};

const void* pair_kernel(int form, int epi);

// Few rows: x on the tensor cores' N side, the weights straight from global memory.
struct StreamParams {
  const void* w;   // bf16 or int8 [R, K], SWIGLU: [2 R, K]
  const void* x;   // bf16 or int8 codes, row t at x + t * x_stride elements
  int64_t x_stride;
  const __nv_bfloat16* x_lo;  // bf16: what x's rounding left, laid out as x, or NULL (not for more than kExactRows rows)
  int T, K, R;
  int swiglu;
  const float* x_scale;  // int8
  const float* w_scale;
  const __nv_bfloat16* addend;
  void* out;
  int out_f32;
  __nv_bfloat16* out_lo;  // bf16 results: what their rounding leaves, or NULL
  __nv_bfloat16* keep;   // SWIGLU: [T, 2 R], or NULL
  int* status;           // the workspace's status words, to be cleared, or NULL
};
constexpr int kStreamRows = 16;  // rows at most
constexpr int kExactRows = 16;
cudaError_t launch_stream(const StreamParams& p, bool int8, bool pdl, int sms, cudaStream_t s);

// Some rows, bf16 or codes as fp16 numbers: the weights on the tensor core's lanes.
struct LaneParams {
  int T, K, R, swiglu;  // as for the stream
  int cols;             // accumulator columns: T, rounded up to 16s
  int split;            // CTAs of a cluster that share a tile's K
  int slots;            // of weights and rows of x, 64 k each or (codes) 128
  int sums_off;         // a tile's sums: behind them, or (0) where they were
  int scale_off;        // the scales
  int stages;           // of widened weights in tensor memory, from this column on
  int stage_at;
  uint32_t idesc;
  const float* x_scale;  // codes
  const float* w_scale;
  const __nv_bfloat16* addend;
  void* out;
  int out_f32;
  __nv_bfloat16* keep;  // bf16 with SWIGLU: [T, 2 R], or NULL
  int pdl;
  int* status;
  int status_keep;
};
constexpr int kLaneRows = 192;  // rows at most
constexpr int lanes_tiles(int R, bool swiglu) { return swiglu ? (R + 63) / 64 : (R + 127) / 128; }
// pdl: behind a launch that writes no weights and lets this one start when all before it have ended.
cudaError_t launch_lanes(LaneParams p, bool int8, const CUtensorMap& w, const CUtensorMap& x, int dev, int smem, int sms, cudaStream_t s);

// codes of rows, as int8 or (half) as fp16 numbers
cudaError_t launch_quantise(int dtype, const void* x, int64_t x_stride, int64_t rows, int inner, void* codes, bool half,
                            float* scale, bool pdl, cudaStream_t s);
// int8 -> fp16, 16 at a time; row r of src at src + r * stride
cudaError_t launch_widen(const int8_t* src, int64_t stride, int64_t rows, int cols, __half* dst, bool pdl, cudaStream_t s);
cudaError_t launch_zero(void* p, int64_t bytes, cudaStream_t s);

}  // namespace dense
}  // namespace moe
