// Launch parameters and constants of the many-row operators, shared by the host
// code (rows_api.cu) and the kernels.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <vector_functions.h>
#include <cstdint>

#include "moe_params.h"

namespace moe {
namespace rows {

constexpr int kMaxN = 256;        // rows of x per tile
constexpr int kMaxStages = 48;    // operand stages in shared memory
constexpr int kMaxRaw = 8;        // slots of quantised codes
constexpr int kWidenThreads = 256;
constexpr int kMaxGroups = 1024 + 8;  // experts and shared experts, or adapters
constexpr int kMaxAdapters = 1024;
constexpr int kMaxSms = 512;      // status words of a launch (two launches': the 4096 bytes of the header)
constexpr uint32_t kWaitLimit = 1u << 21;
constexpr unsigned long long kDrainNs = 1000000ull;

// What the epilogue makes of the accumulators.
enum Epi {
  EPI_SWIGLU = 0,  // bf16 silu(gate) * up
  EPI_F32 = 1,     // fp32
  EPI_BF16 = 2,    // bf16
  EPI_TWO = 3      // the sum of two bf16 numbers, with a scale per group (bf16 weights)
};

// How the rows' adapters join the sum.
enum AdMode {
  AD_NONE = 0,
  AD_STEPS = 1,    // more K steps on the tensor core, each over one adapter's rows
  AD_EPILOGUE = 2  // fp32 products of few rows, added in the epilogue
};

__host__ __device__ constexpr int epilogue_warps(int fmt) { return 8; }
// Accumulators at once: two while tensor memory (512 columns) has room for them, beside
// the widened weights of a quantised format.
__host__ __device__ constexpr int acc_buffers(int fmt, int nmax) {
  return 4 * nmax <= (fmt == FMT_BF16 ? 512 : 128) ? 2 : 1;
}
// Steps of 64 k in a stage.
__host__ __device__ constexpr int stage_steps(int fmt) { return fmt == FMT_BF16 ? 1 : 2; }
constexpr int threads_of(int fmt) {
  return 128 + 32 * epilogue_warps(fmt) + (fmt == FMT_BF16 ? 0 : kWidenThreads);
}
// k's in 128 bytes of codes
constexpr int kmath(int fmt) { return fmt == FMT_FP8 ? 128 : 256; }

// A tile of a launch with grouped rows: `n` rows of `group` from position p0 on, the
// block-th of the group's `blocks` tiles. Block and count have a word each (a group of
// 2^24 rows has more than 2^16 tiles); group and rows share one.
constexpr int kTileGroupBits = 16;
static_assert(kMaxGroups <= 1 << kTileGroupBits && kMaxN < 1 << (31 - kTileGroupBits), "a tile's group and rows share a word");
__host__ __device__ inline int4 pack_tile(int group, int p0, int n, int block, int blocks) {
  return make_int4(group | n << kTileGroupBits, p0, block, blocks);
}
__host__ __device__ inline int tile_group(const int4& t) { return t.x & ((1 << kTileGroupBits) - 1); }
__host__ __device__ inline int tile_rows(const int4& t) { return t.x >> kTileGroupBits; }
__host__ __device__ inline int tile_first(const int4& t) { return t.y; }
__host__ __device__ inline int tile_block(const int4& t) { return t.z; }
__host__ __device__ inline int tile_blocks(const int4& t) { return t.w; }

struct GemmParams {
  // weights
  int R;            // output rows per group (EPI_SWIGLU: gate rows)
  int K;
  int rt;           // weight rows per sub-tile (multiple of 8, <= 128)
  int nrb;          // tiles along R
  int groups_main;  // groups of map_w; later ones are map_s's
  const void* wscale;    // FP8 / NVFP4 block scales
  const void* wscale_s;
  const float* gscale;   // NVFP4 tensor scales; EPI_TWO: a scale per group
  const float* gscale_s;
  // rows of x (map_x)
  const int* src_row;  // row at each sorted position (NULL: the position)
  int box_rows;        // without a list: rows of a copy (map_x's box)
  int all_rows;        // rows of each group from groups_main on, read through map_u; 0: as the others
  int all_first;       // the first such group's first position
  int rows;            // uniform tiles: rows in all
  int nmax;            // rows per tile at most
  const int4* ents;    // pack_tile's, or NULL: uniform tiles
  const int* nent;
  // adapters
  int ad_mode;         // AdMode
  int num_adapters;
  int rank;
  // AD_STEPS: positions off[a] .. off[a + 1] (multiples of 16) belong to adapter a,
  // off[num_adapters] .. off[num_adapters + 1] to none; B is map_s
  const int* adapter_off;
  // and the rows' products A x are map_u's, [positions, 2 rank]: hi, then lo
  // AD_EPILOGUE: rows in their own order
  const int* ids;
  const float* u32;        // [rows, rank]
  const __nv_bfloat16* b;  // [num_adapters][halves * R][rank]
  int ad_off;              // shared memory of the tile's adapter products
  // results
  void* out;
  int64_t out_stride;
  const int* out_row;  // row of out at each sorted position (NULL: the position)
  const __nv_bfloat16* addend;  // laid out as out
  int lo_off;          // EPI_TWO: columns from a result to what its rounding left
  int* status;         // [kMaxSms] one word per CTA: 1 = a wait ran into its limit
  int* status_clear;   // [kMaxSms] another launch's words when that launch is left out, or NULL
  int status_keep;     // 1: a later round of the same call; words are only set
  // shared memory
  int stages;
  int stage_bytes;
  int raw_off;
  int raw_slots;
  int pdl;
  int split;  // CTAs of a cluster that share a tile's K (bf16 weights, uniform tiles, no AD_STEPS)
};

const void* gemm_kernel(int epi, int fmt);
}  // namespace rows
}  // namespace moe
