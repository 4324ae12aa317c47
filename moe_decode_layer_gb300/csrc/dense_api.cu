// Host side of the dense operators: checks, workspace layout, launch shapes.
// See include/moe_decode_dense.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "../../include/moe_decode_dense.h"
#include "dense_params.h"
#include "rows_host.h"

using namespace moe;
using namespace moe::rows;
using namespace moe::dense;

namespace {

constexpr int kMostWidth = 65536;
constexpr size_t kStatusBytes = kStatusKernels * kMaxSms * 4;
static_assert(lanes_tiles(kMostWidth, true) <= kStatusKernels * kMaxSms, "a CTA of the widest product has a status word");

// [halves][rows][cols] of 2-byte numbers (or fp32, or codes), copied in boxes of 128 bytes x box_rows rows;
// what lies past the matrix reads as zero and is not written.
bool make_map(CUtensorMap* m, const void* ptr, int64_t pitch, int64_t cols, int64_t rows, int box_rows, int halves = 1,
              int64_t half_bytes = 0, bool f32 = false, bool codes = false) {
  EncodeTiled enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)halves};
  const cuuint64_t strides[2] = {(cuuint64_t)pitch, (cuuint64_t)(halves > 1 ? half_bytes : pitch)};
  const cuuint32_t box[3] = {f32 ? 32u : codes ? 128u : 64u, (cuuint32_t)box_rows, 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return enc(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
             3, const_cast<void*>(ptr), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A matrix operand: a stored matrix [rows][cols], and whether its rows or its columns are k's.
struct Matrix {
  const void* ptr;
  int64_t pitch;  // bytes
  int64_t rows, cols;
};

PairParams one_pass() {
  PairParams p = {};
  p.passes = 1;
  return p;
}

struct PairLaunch {
  PairParams p = one_pass();
  CUtensorMap a, b, d, e, g, d2;
  int form = 0, epi = 0;
};

// Width of the tiles and pairs that share a tile's K. A step of 64 k costs its tensor time (2 bn
// clocks), its operand bytes (about 55 a clock and SM from L2) and, where few row tiles share
// the columns' operand, that operand's bytes at an SM's share of the HBM rate (23 a clock; at
// most 45 for an SM while others rest); a tile about 2500 clocks of start and epilogue, 1800
// more where sums are joined. Clusters of four and eight CTAs do not fill every SM: of 152, 36 and 15
// are resident at once (a 16th of eight waited for another's end: 34 us for a product of 256 rows
// that takes 12).
void shape_of(PairParams& p, bool swiglu, const Device& d) {
  const int pairs = d.sms / 2, ksteps = (p.K + 63) / 64 * p.passes;
  double least = 1e300;
  p.tiles_m = (int)cdiv(p.M, kTileM);
  p.tiles_m2 = (int)cdiv(p.M2, kTileM);
  for (int bn : {256, 192, 128})
    for (int split : {1, 2, 4}) {
      if (swiglu && bn == 192) continue;
      const int tiles_n = (int)cdiv(p.N, swiglu ? bn / 2 : bn);
      const int tiles_n2 = (int)cdiv(p.N2, bn);
      const int64_t tiles = (int64_t)p.tiles_m * tiles_n + (int64_t)p.tiles_m2 * tiles_n2;
      if (split > 1 && (tiles > (split == 2 ? d.sms * 9 / 38 : d.sms / 10) || ksteps < 4 * split)) continue;
      const double waves = split > 1 ? 1 : (double)cdiv(tiles, pairs);
      const double ctas = 2.0 * std::min<double>((double)tiles * split, pairs);
      const double rows = std::min(128.0, std::max(16.0, p.M / 2.0));
      const double hbm = bn * 64.0 / (std::min(45.0, 23.0 * d.sms / ctas) * std::min(p.tiles_m, kGroupM));
      const double step = std::max({2.0 * bn, (rows * 128.0 + bn * 64.0) / 55.0, hbm});
      const double cost = waves * (cdiv(ksteps, split) * step + 600.0) + 2500.0 + (split > 1 ? 1800.0 : 0.0);
      if (cost < least * 0.98) {
        least = cost;
        p.bn = bn;
        p.split = split;
        p.tiles_n = tiles_n;
        p.tiles_n2 = tiles_n2;
      }
    }
}

constexpr int kFewWarpsK = 512;

// Operands a and b, and results: map d at `out` (and e, g as the epilogue has them). Descriptors only.
bool prepare(PairLaunch& l, int form, int epi, const Matrix& a, const Matrix& b, bool fp16, const Device& d) {
  PairParams& p = l.p;
  const bool swiglu = epi == PAIR_SWIGLU || epi == PAIR_SWIGLU_F32, codes = form == FORM_KK8;
  l.form = form;
  l.epi = epi;
  shape_of(p, swiglu, d);
  p.bufs = epi == PAIR_DSWIGLU_LO ? 6 : epi == PAIR_DSWIGLU || (epi == PAIR_SWIGLU && p.keep) ? 3 : epi == PAIR_SWIGLU || codes ? 1 : 2;
  // (A copy takes the TMA unit about two clocks a row of 128 bytes, also of rows that it fills with zeros.)
  const int a_rows = form != FORM_MM && p.M <= 128 ? (int)up(p.M, 8) : 128;
  const int b_bytes = form == FORM_KK || codes ? p.bn * 64 : (int)cdiv(p.bn, 128) * 8192;
  p.a_bytes = a_rows * 128;
  p.stage_bytes = p.a_bytes + b_bytes;
  p.step_bytes = (a_rows < 128 ? 1 : 2) * p.a_bytes + (codes ? 0 : 2 * b_bytes);
  // The boxes of eight warps leave four or five stages of 256 columns, those of four one more. Where a
  // tile's product is long enough for its epilogue, that is faster (the round of a stage's barriers and
  // copies takes about 2600 clocks).
  p.ewarps = codes || epi == PAIR_DSWIGLU_LO || (p.split == 1 && p.K >= kFewWarpsK) ? 4 : 8;
  const int end = d.smem - 2048;
  p.scale_off = end - 4096;
  int room = end - p.ewarps * p.bufs * kStageBox - (codes ? 4096 : 0);
  p.raw_slots = 0;
  if (codes) {
    // the copies in flight are the slots of codes: four at least, and up to six stages
    p.stages = std::min(6, (room - 4 * p.bn * 64) / p.stage_bytes);
    p.raw_slots = std::min(kRawSlots, (room - p.stages * p.stage_bytes) / (p.bn * 64)) & ~1;
    p.raw_off = p.stages * p.stage_bytes;
  } else {
    p.stages = std::min(kPairStages, room / p.stage_bytes);
  }
  p.ahead = p.tiles_m <= 2 && form != FORM_MM && (codes || a_rows == 128) ? 8 : 0;
  // fp32 accumulators; bf16 or fp16 operands; k or the operand's own index innermost; M = 256 of a pair
  p.idesc = 1u << 4 | (fp16 ? 0u : 1u << 7 | 1u << 10) | (form == FORM_MM ? 1u << 15 : 0u) |
            (form == FORM_KM || form == FORM_MM ? 1u << 16 : 0u) | (uint32_t)(p.bn >> 3) << 17 | 16u << 24;
  const bool ok_a = make_map(&l.a, a.ptr, a.pitch, a.cols, a.rows, form == FORM_MM ? 64 : a_rows);
  const bool ok_b = swiglu ? make_map(&l.b, b.ptr, b.pitch, b.cols, b.rows / 2, p.bn / 2, 2, b.pitch * (b.rows / 2), false, codes)
                           : make_map(&l.b, b.ptr, b.pitch, b.cols, b.rows, form == FORM_KK || codes ? p.bn / 2 : 64, 1, 0, false, codes);
  l.e = l.g = l.d2 = l.a;
  p.box_off = std::max(p.stages * p.stage_bytes + p.raw_slots * p.bn * 64, p.split > 1 ? p.bn * 512 : 0);
  return ok_a && ok_b && p.stages >= 2 && (!codes || (p.raw_slots >= 2 && p.stages >= 3)) && p.box_off + p.ewarps * p.bufs * kStageBox <= (codes ? p.scale_off : end);
}

bool out_map(CUtensorMap* m, const void* out, int64_t M, int64_t N, bool f32, bool reduce) {
  if (f32 && reduce) return make_map(m, out, N * 4, N, M, 32, 1, 0, true);
  // an fp32 column counts as two
  return make_map(m, out, N * (f32 ? 4 : 2), N * (f32 ? 2 : 1), M, 32);
}

// A second product of FORM_MM, which p.M2 and p.N2 have announced.
bool prepare_second(PairLaunch& l, const Matrix& a, const Matrix& b, const void* out, bool f32) {
  return make_map(&l.e, a.ptr, a.pitch, a.cols, a.rows, 64) && make_map(&l.g, b.ptr, b.pitch, b.cols, b.rows, 64) &&
         out_map(&l.d2, out, l.p.M2, l.p.N2, f32, l.p.reduce);
}

// Results [M, N] of 2 bytes, or fp32 (as pairs of 2 bytes where nothing is added), and their addends.
bool prepare_out(PairLaunch& l, const void* out, bool f32) {
  const PairParams& p = l.p;
  if (p.addend && l.epi == PAIR_BF16 && !make_map(&l.g, p.addend, (int64_t)p.N * 2, p.N, p.M, 32)) return false;
  return out_map(&l.d, out, p.M, p.N, f32, p.reduce);
}

cudaError_t launch(PairLaunch& l, const Device& d, bool pdl, cudaStream_t s) {
  const void* k = pair_kernel(l.form, l.epi);
  static std::atomic<uint64_t> ready[4][PAIR_DSWIGLU_LO + 1];  // per kernel: devices whose limit is set
  if (d.id >= 64 || !(ready[l.form][l.epi].load() >> d.id & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, d.smem - 1024);
    if (e != cudaSuccess) return e;
    if (d.id < 64) ready[l.form][l.epi].fetch_or(1ull << d.id);
  }
  l.p.pdl = pdl;
  const int64_t tiles = (int64_t)l.p.tiles_m * l.p.tiles_n + (int64_t)l.p.tiles_m2 * l.p.tiles_n2;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)(2 * l.p.split * (l.p.split > 1 ? tiles : std::min<int64_t>(tiles, d.sms / 2))));
  c.blockDim = dim3(pair_threads(l.form));
  // All of the SM's shared memory: a CTA takes all tensor memory, and a pair's CTAs wait for one
  // another, so none may wait for tensor memory that a CTA of another launch on its SM holds.
  c.dynamicSmemBytes = d.smem - 1024;
  c.stream = s;
  cudaLaunchAttribute a[2];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  a[1].id = cudaLaunchAttributeClusterDimension;
  a[1].val.clusterDim.x = 2 * l.p.split;
  a[1].val.clusterDim.y = a[1].val.clusterDim.z = 1;
  c.attrs = a;
  c.numAttrs = 2;
  void* args[] = {&l.p, &l.a, &l.b, &l.d, &l.e, &l.g, &l.d2};
  return cudaLaunchKernelExC(&c, k, args);
}

// Places in a workspace, 256 bytes apart at least.
struct Places {
  size_t at = 0;
  size_t take(size_t bytes) {
    const size_t o = at;
    at = up(at + bytes, 256);
    return o;
  }
};

// Rows of bf16: few take a stream of the weights, 8 or, where these are small, 16 (16 rows of the 1024 x 2048 block
// 10.1 us, on the lanes 11.2; 4096 x 8192 45.0, and 37.8 on the lanes); up to 128 have the weights on the lanes (64 rows, 4096 x
// 8192 and 2560 x 6912: 41.7 and 30.6 us, 49.3 and 34.8 in pairs; 128: 47.0 and 35.0, 52.6 and 37.2); more take the pair product.
constexpr int64_t kStreamBytes = 16 << 20;
bool few(int64_t rows, int64_t bytes) { return rows <= 8 || (rows <= kStreamRows && bytes <= kStreamBytes); }
// Codes: a stream up to 8 rows, or 16 where the weights on the lanes are few tiles and their start and end count (16 rows,
// 4096 to 2 x 8192: 21.4 us and 18.9, 8192 to 4096: 11.4 and 14.3). These up to 128 rows, or 192 where the
// pair product has few tiles as well (160 rows, 8192 to 4096: 22.2 us and 30.4 in pairs, 192: 23.0 and 30.4;
// 4096 to 2 x 8192: 128 rows 27.1 and 31.5, 160 30.7 and 31.7).
constexpr int kFewTiles = 76, kLanesAlways = 128;
bool few_tiles(const moe_int8_config& c) { return lanes_tiles(c.outer, c.swiglu) <= kFewTiles; }
bool few_codes(int64_t rows, const moe_int8_config& c) {
  return rows <= 8 || (rows <= 16 && few_tiles(c));
}
bool on_lanes(int64_t rows, const moe_int8_config& c) { return !few_codes(rows, c) && rows <= (few_tiles(c) ? kLaneRows : kLanesAlways); }

// ------------------------------------------------------------------ int8
moe_status check_int8(const moe_int8_config* c) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (c->inner <= 0 || c->outer <= 0) return MOE_ERR_INVALID_ARG;
  if (c->x_dtype != MOE_I8 && c->x_dtype != MOE_BF16 && c->x_dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (c->out_dtype != MOE_BF16 && c->out_dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (c->inner % 16 || c->outer % 8 || c->inner > kMostWidth || c->outer > kMostWidth) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

struct Int8Plan {
  size_t status, codes, scale, bytes;
};
// A stream takes the codes as they are, the pair product fp16 copies.
Int8Plan int8_plan(const moe_int8_config& c, int64_t rows) {
  Places pl;
  Int8Plan p = {};
  const bool made = c.x_dtype != MOE_I8;
  if (few_codes(rows, c) && !made) return p;  // nothing is kept, and nothing waits
  p.status = pl.take(kStatusBytes);
  p.codes = pl.take((size_t)rows * c.inner * (few_codes(rows, c) ? 1 : 2));
  if (made) p.scale = pl.take((size_t)rows * 4);
  p.bytes = pl.at;
  return p;
}

// A product of codes (or of what is quantised first) with one matrix; descriptors in l before any launch.
struct Int8Product {
  moe_int8_config c;
  const int8_t* w;
  const float* w_scale;
  const void* x;
  const float* x_scale;  // MOE_I8
  int64_t x_stride;
  const void* addend;
  void* out;
  int64_t rows;
  // in the workspace
  int* status;
  bool status_keep;
  uint8_t* codes;
  float* scale;
  PairLaunch l;
};

moe_status prepare_int8(Int8Product& a, const Device& d) {
  if (few_codes(a.rows, a.c)) return MOE_OK;
  const bool f32 = a.c.out_dtype == MOE_F32;
  PairParams& p = a.l.p;
  p.M = (int)a.rows;
  p.N = a.c.outer;
  p.K = a.c.inner;
  p.row_scale = a.c.x_dtype == MOE_I8 ? a.x_scale : a.scale;
  p.col_scale = a.w_scale;
  p.addend = static_cast<const __nv_bfloat16*>(a.addend);
  p.status = a.status;
  p.status_keep = a.status_keep;
  const int64_t k = a.c.inner, w_rows = (int64_t)a.c.outer * (a.c.swiglu ? 2 : 1);
  if (on_lanes(a.rows, a.c)) {
    const int64_t halves = a.c.swiglu ? 2 : 1;
    return make_map(&a.l.b, a.w, k, k, a.c.outer, 64, (int)halves, k * a.c.outer, false, true) &&
                   make_map(&a.l.a, a.codes, k * 2, k, a.rows, (int)up(a.rows, 16))
               ? MOE_OK
               : MOE_ERR_CUDA;
  }
  const int epi = a.c.swiglu ? (f32 ? PAIR_SWIGLU_F32 : PAIR_SWIGLU) : f32 ? PAIR_F32 : PAIR_BF16;
  return prepare(a.l, FORM_KK8, epi, {a.codes, k * 2, a.rows, k}, {a.w, k, w_rows, k}, true, d) && prepare_out(a.l, a.out, f32)
             ? MOE_OK
             : MOE_ERR_CUDA;
}

cudaError_t launch_int8(Int8Product& a, const Device& d, bool pdl, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  const bool made = a.c.x_dtype != MOE_I8, small = few_codes(a.rows, a.c);
  if (made)
    e = launch_quantise(a.c.x_dtype, a.x, a.x_stride, a.rows, a.c.inner, a.codes, !small, a.scale, pdl, s);
  else if (!small)
    e = launch_widen(static_cast<const int8_t*>(a.x), a.x_stride, a.rows, a.c.inner, reinterpret_cast<__half*>(a.codes), pdl, s);
  if (e != cudaSuccess) return e;
  pdl = pdl || made || !small;
  if (on_lanes(a.rows, a.c)) {
    LaneParams p = {};
    p.T = (int)a.rows;
    p.K = a.c.inner;
    p.R = a.c.outer;
    p.swiglu = a.c.swiglu;
    p.cols = (int)up(a.rows, 16);
    p.x_scale = a.l.p.row_scale;
    p.w_scale = a.w_scale;
    p.addend = a.l.p.addend;
    p.out = a.out;
    p.out_f32 = a.c.out_dtype == MOE_F32;
    p.status = a.status;
    p.status_keep = a.status_keep;
    p.pdl = 1;
    return launch_lanes(p, true, a.l.b, a.l.a, d.id, d.smem, d.sms, s);
  }
  if (!small) return launch(a.l, d, pdl, s);
  StreamParams p = {};
  p.w = a.w;
  p.x = made ? static_cast<const void*>(a.codes) : a.x;
  p.x_stride = made ? a.c.inner : a.x_stride;
  p.T = (int)a.rows;
  p.K = a.c.inner;
  p.R = a.c.outer;
  p.swiglu = a.c.swiglu != 0;
  p.x_scale = made ? a.scale : a.x_scale;
  p.w_scale = a.w_scale;
  p.addend = static_cast<const __nv_bfloat16*>(a.addend);
  p.out = a.out;
  p.out_f32 = a.c.out_dtype == MOE_F32;
  p.status = a.status_keep ? nullptr : a.status;
  return launch_stream(p, true, pdl, d.sms, s);
}

// ------------------------------------------------------------------ feed-forward
moe_status check_ff(const moe_ff_config* c) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (c->hidden <= 0 || c->inter <= 0) return MOE_ERR_INVALID_ARG;
  if (c->wdtype != MOE_W_BF16 && c->wdtype != MOE_W_INT8) return MOE_ERR_UNSUPPORTED;
  const int step = c->wdtype == MOE_W_INT8 ? 16 : 8;
  if (c->hidden % step || c->inter % step || c->hidden > kMostWidth || c->inter > kMostWidth) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// A handful of rows in bf16: h as the sum of two bf16 numbers. It costs a stream little (one row, 4096 x 8192:
// 33.3 -> 34.6 us), and so the result has its own rounding alone. h's rounding counts as much in many rows: the
// limit is where the cost shows. More rows of large matrices read twice the rows of h for every weight (8 rows: 35 -> 40 us)
// and do without.
constexpr int64_t kAlwaysExact = 4;
bool exact(int64_t rows, const moe_ff_config& c) {
  return c.wdtype == MOE_W_BF16 && (rows <= kAlwaysExact || (rows <= kExactRows && (int64_t)c.hidden * c.inter * 4 <= kStreamBytes));
}

struct FfPlan {
  size_t status, h, codes, scale, bytes;
};
FfPlan ff_plan(const moe_ff_config& c, int64_t rows) {
  Places pl;
  FfPlan p = {};
  p.status = pl.take(kStatusBytes);
  const bool int8 = c.wdtype == MOE_W_INT8;
  p.h = pl.take((size_t)rows * c.inter * (int8 || exact(rows, c) ? 4 : 2));
  if (int8) {
    // (both products' rows in turn; a stream takes a byte each)
    p.codes = pl.take((size_t)rows * std::max(c.hidden, c.inter) * 2);
    p.scale = pl.take((size_t)rows * 4);
  }
  p.bytes = pl.at;
  return p;
}

struct BackwardPlan {
  size_t status, both, h, bytes;
};
// A few rows of a narrow block: dg, du and h as two bf16 numbers each, side by side in a row. With one number a gradient
// of many values is 1.41 times its own rounding off (root mean square); that of few varies from input to input (1.9 times in
// the largest seen, which is no bound). dx's product is then twice as long and the weight gradients have a step more: one
// row, 1024 x 2048, 38 us and 32 without. The limit is where that cost is a fixed few microseconds.
constexpr int64_t kExactValues = 4096;
int64_t exact_backward_rows(const moe_ff_config& c) {
  return (int64_t)c.hidden * c.inter * 4 <= kStreamBytes ? kExactValues / std::min(c.hidden, c.inter) : 0;
}
bool exact_backward(int64_t rows, const moe_ff_config& c) { return rows <= exact_backward_rows(c); }
BackwardPlan backward_plan(const moe_ff_config& c, int64_t rows) {
  Places pl;
  BackwardPlan p = {};
  const size_t each = exact_backward(rows, c) ? 2 : 1;
  p.status = pl.take(kStatusBytes);
  p.both = pl.take((size_t)rows * c.inter * 4 * each);
  p.h = pl.take((size_t)rows * c.inter * 2 * each);
  p.bytes = pl.at;
  return p;
}

// Byte ranges of a call.
struct Range {
  const void* ptr;
  int64_t bytes;
};
bool any_overlap(const Range& a, std::initializer_list<Range> others) {
  for (const Range& o : others)
    if (overlap(a.ptr, a.bytes, o.ptr, o.bytes)) return true;
  return false;
}

}  // namespace

extern "C" {

moe_status moe_decode_quantise(int32_t dtype, int32_t inner, const void* x, int64_t x_stride, int64_t rows, int8_t* codes,
                               float* scale, moe_stream_t stream) {
  if (inner <= 0 || rows < 0 || rows > kMaxRows) return MOE_ERR_INVALID_ARG;
  if ((dtype != MOE_BF16 && dtype != MOE_F32) || inner % 8 || inner > kMostWidth) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  const int64_t size = dtype == MOE_F32 ? 4 : 2;
  if (!x || !codes || !scale || !aligned16(x) || !aligned16(codes) || !aligned4(scale)) return MOE_ERR_INVALID_ARG;
  if (x_stride < inner || x_stride * size % 16) return MOE_ERR_INVALID_ARG;
  if (rows_overlap(x, x_stride * size, inner * size, rows, codes, rows * inner) ||
      rows_overlap(x, x_stride * size, inner * size, rows, scale, rows * 4) || overlap(codes, rows * inner, scale, rows * 4))
    return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_quantise(dtype, x, x_stride, rows, inner, codes, false, scale, false,
                                     reinterpret_cast<cudaStream_t>(stream)));
}

moe_status moe_decode_project_int8_check(const moe_int8_config* c) { return check_int8(c); }

moe_status moe_decode_project_int8_workspace(const moe_int8_config* c, int64_t rows, size_t* bytes) {
  const moe_status st = check_int8(c);
  if (st != MOE_OK) return st;
  if (!bytes || rows < 0 || rows > kMaxRows) return MOE_ERR_INVALID_ARG;
  *bytes = rows ? int8_plan(*c, rows).bytes : 0;
  return MOE_OK;
}

moe_status moe_decode_project_int8(const moe_int8_config* c, const int8_t* w, const float* w_scale, const void* x,
                                   const float* x_scale, int64_t x_stride, const void* addend, void* out, int64_t rows,
                                   void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  moe_status st = check_int8(c);
  if (st != MOE_OK) return st;
  if (rows < 0 || rows > kMaxRows) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  const bool codes = c->x_dtype == MOE_I8, f32 = c->out_dtype == MOE_F32;
  const int64_t size = codes ? 1 : c->x_dtype == MOE_F32 ? 4 : 2;
  if (!w || !w_scale || !x || !out || (codes && !x_scale)) return MOE_ERR_INVALID_ARG;
  if (c->swiglu && addend) return MOE_ERR_INVALID_ARG;
  if (!aligned16(w) || !aligned16(w_scale) || !aligned16(x) || !aligned16(addend) || !aligned16(out) || !aligned16(workspace))
    return MOE_ERR_INVALID_ARG;
  if (codes && !aligned4(x_scale)) return MOE_ERR_INVALID_ARG;
  if (x_stride < c->inner || x_stride * size % 16) return MOE_ERR_INVALID_ARG;
  const int64_t add_bytes = rows * c->outer * 2, out_bytes = f32 ? 2 * add_bytes : add_bytes;
  if (rows_overlap(x, x_stride * size, c->inner * size, rows, out, out_bytes)) return MOE_ERR_INVALID_ARG;
  if (codes && overlap(x_scale, rows * 4, out, out_bytes)) return MOE_ERR_INVALID_ARG;
  if ((addend != out || f32) && overlap(addend, add_bytes, out, out_bytes)) return MOE_ERR_INVALID_ARG;
  const int64_t w_rows = (int64_t)c->outer * (c->swiglu ? 2 : 1);
  if (any_overlap({out, out_bytes}, {{w, w_rows * c->inner}, {w_scale, w_rows * 4}})) return MOE_ERR_INVALID_ARG;
  const Int8Plan p = int8_plan(*c, rows);
  if (workspace_bytes < p.bytes || (p.bytes && !workspace)) return MOE_ERR_INVALID_ARG;
  Device d;
  if (!device(&d)) return MOE_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  Int8Product a = {*c,  w,    w_scale, x, x_scale, x_stride, addend, out, rows,
                   workspace && workspace_bytes >= kStatusBytes ? reinterpret_cast<int*>(ws + p.status) : nullptr, false,
                   ws + p.codes, reinterpret_cast<float*>(ws + p.scale), {}};
  st = prepare_int8(a, d);
  if (st != MOE_OK) return st;
  return cuda_status(launch_int8(a, d, false, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status moe_decode_ff_check(const moe_ff_config* c) { return check_ff(c); }

moe_status moe_decode_ff_workspace(const moe_ff_config* c, int64_t rows, size_t* bytes) {
  const moe_status st = check_ff(c);
  if (st != MOE_OK) return st;
  if (!bytes || rows < 0 || rows > kMaxRows) return MOE_ERR_INVALID_ARG;
  *bytes = 0;  // (fewer rows may need more: h as two numbers)
  for (int64_t r : {rows, std::min<int64_t>(rows, kAlwaysExact), std::min<int64_t>(rows, kExactRows)})
    if (r) *bytes = std::max(*bytes, ff_plan(*c, r).bytes);
  return MOE_OK;
}

moe_status moe_decode_ff(const moe_ff_config* c, const moe_ff_weights* wt, const void* x, int64_t x_stride,
                         const void* residual, void* gate_up, void* out, int64_t rows, void* workspace,
                         size_t workspace_bytes, moe_stream_t stream) {
  moe_status st = check_ff(c);
  if (st != MOE_OK) return st;
  if (rows < 0 || rows > kMaxRows) return MOE_ERR_INVALID_ARG;
  const bool int8 = c->wdtype == MOE_W_INT8;
  if (int8 && gate_up) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!wt || !wt->w13 || !wt->w2 || !x || !out || !workspace || (int8 && (!wt->s13 || !wt->s2))) return MOE_ERR_INVALID_ARG;
  if (!aligned16(wt->w13) || !aligned16(wt->w2) || !aligned16(x) || !aligned16(residual) || !aligned16(gate_up) ||
      !aligned16(out) || !aligned16(workspace) || (int8 && (!aligned16(wt->s13) || !aligned16(wt->s2))))
    return MOE_ERR_INVALID_ARG;
  if (x_stride < c->hidden || x_stride % 8) return MOE_ERR_INVALID_ARG;
  // The second product, which writes out, starts when the first has read x; each of its
  // results takes its own residual first.
  const int64_t out_bytes = rows * c->hidden * 2, kept_bytes = rows * c->inter * 4;
  if (residual != out && overlap(residual, out_bytes, out, out_bytes)) return MOE_ERR_INVALID_ARG;
  if ((x != out || (x_stride != c->hidden && rows > 1)) && rows_overlap(x, x_stride * 2, c->hidden * 2, rows, out, out_bytes))
    return MOE_ERR_INVALID_ARG;
  const int64_t size = int8 ? 1 : 2, halves = 2 * (int64_t)c->inter;
  for (const Range& o : {Range{out, out_bytes}, Range{gate_up, kept_bytes}})
    if (any_overlap(o, {{wt->w13, halves * c->hidden * size}, {wt->w2, (int64_t)c->hidden * c->inter * size},
                        {int8 ? wt->s13 : nullptr, halves * 4}, {int8 ? wt->s2 : nullptr, (int64_t)c->hidden * 4}}))
      return MOE_ERR_INVALID_ARG;
  if (gate_up && (rows_overlap(x, x_stride * 2, c->hidden * 2, rows, gate_up, kept_bytes) ||
                  any_overlap({gate_up, kept_bytes}, {{residual, out_bytes}, {out, out_bytes}})))
    return MOE_ERR_INVALID_ARG;
  const FfPlan p = ff_plan(*c, rows);
  if (workspace_bytes < p.bytes) return MOE_ERR_INVALID_ARG;
  Device d;
  if (!device(&d)) return MOE_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int* status = reinterpret_cast<int*>(ws + p.status);
  void* h = ws + p.h;
  const int64_t hid = c->hidden, in = c->inter;

  if (int8) {
    uint8_t* codes = ws + p.codes;
    float* scale = reinterpret_cast<float*>(ws + p.scale);
    Int8Product one = {{c->hidden, c->inter, 1, MOE_BF16, MOE_F32}, static_cast<const int8_t*>(wt->w13), wt->s13, x, nullptr,
                       x_stride, nullptr, h, rows, status, false, codes, scale, {}};
    Int8Product two = {{c->inter, c->hidden, 0, MOE_F32, MOE_BF16}, static_cast<const int8_t*>(wt->w2), wt->s2, h, nullptr,
                       in, residual, out, rows, status, true, codes, scale, {}};
    if ((st = prepare_int8(one, d)) != MOE_OK || (st = prepare_int8(two, d)) != MOE_OK) return st;
    const cudaError_t e = launch_int8(one, d, false, s);
    return cuda_status(e == cudaSuccess ? launch_int8(two, d, true, s) : e);
  }

  if (few(rows, hid * in * 4)) {
    StreamParams one = {}, two = {};
    one.w = wt->w13;
    one.x = x;
    one.x_stride = x_stride;
    one.T = two.T = (int)rows;
    one.K = two.R = c->hidden;
    one.R = two.K = c->inter;
    one.swiglu = 1;
    one.keep = static_cast<__nv_bfloat16*>(gate_up);
    one.out = h;
    one.status = status;
    if (exact(rows, *c)) {
      one.out_lo = static_cast<__nv_bfloat16*>(h) + rows * in;
      two.x_lo = one.out_lo;
    }
    two.w = wt->w2;
    two.x = h;
    two.x_stride = in;
    two.addend = static_cast<const __nv_bfloat16*>(residual);
    two.out = out;
    const cudaError_t e = launch_stream(one, false, false, d.sms, s);
    return cuda_status(e == cudaSuccess ? launch_stream(two, false, true, d.sms, s) : e);
  }

  if (rows <= kLanesAlways) {
    LaneParams one = {}, two = {};
    CUtensorMap w1, x1, w2, x2;
    one.T = two.T = (int)rows;
    one.cols = two.cols = (int)up(rows, 16);
    one.K = two.R = c->hidden;
    one.R = two.K = c->inter;
    one.swiglu = two.pdl = two.status_keep = 1;
    one.out = h;
    one.keep = static_cast<__nv_bfloat16*>(gate_up);
    two.addend = static_cast<const __nv_bfloat16*>(residual);
    two.out = out;
    one.status = two.status = status;
    if (!make_map(&w1, wt->w13, hid * 2, hid, in, 64, 2, in * hid * 2) || !make_map(&x1, x, x_stride * 2, hid, rows, one.cols) ||
        !make_map(&w2, wt->w2, in * 2, in, hid, 64) || !make_map(&x2, h, in * 2, in, rows, one.cols))
      return MOE_ERR_CUDA;
    const cudaError_t e = launch_lanes(one, false, w1, x1, d.id, d.smem, d.sms, s);
    return cuda_status(e == cudaSuccess ? launch_lanes(two, false, w2, x2, d.id, d.smem, d.sms, s) : e);
  }

  PairLaunch one, two;
  one.p.M = two.p.M = (int)rows;
  one.p.N = two.p.K = c->inter;
  one.p.K = two.p.N = c->hidden;
  one.p.keep = gate_up != nullptr;
  two.p.addend = static_cast<const __nv_bfloat16*>(residual);
  one.p.status = two.p.status = status;
  two.p.status_keep = 1;
  if (!prepare(one, FORM_KK, PAIR_SWIGLU, {x, x_stride * 2, rows, hid}, {wt->w13, hid * 2, 2 * in, hid}, false, d) ||
      !prepare_out(one, h, false) ||
      (gate_up && !make_map(&one.e, gate_up, in * 4, in, rows, 32, 2, in * 2)) ||
      !prepare(two, FORM_KK, PAIR_BF16, {h, in * 2, rows, in}, {wt->w2, in * 2, hid, in}, false, d) ||
      !prepare_out(two, out, false))
    return MOE_ERR_CUDA;
  const cudaError_t e = launch(one, d, false, s);
  return cuda_status(e == cudaSuccess ? launch(two, d, true, s) : e);
}

moe_status moe_decode_ff_backward_workspace(const moe_ff_config* c, int64_t rows, size_t* bytes) {
  const moe_status st = check_ff(c);
  if (st != MOE_OK) return st;
  if (c->wdtype != MOE_W_BF16) return MOE_ERR_UNSUPPORTED;
  if (!bytes || rows < 0 || rows > kMaxRows) return MOE_ERR_INVALID_ARG;
  *bytes = 0;  // (fewer rows may need more)
  for (int64_t r : {rows, std::min(rows, exact_backward_rows(*c))})
    if (r) *bytes = std::max(*bytes, backward_plan(*c, r).bytes);
  return MOE_OK;
}

moe_status moe_decode_ff_backward(const moe_ff_config* c, const moe_ff_weights* wt, const void* grad, int64_t grad_stride,
                                  const void* x, int64_t x_stride, const void* gate_up, void* dx, void* dw13, void* dw2,
                                  int32_t dw_dtype, int32_t accumulate, int64_t rows, void* workspace,
                                  size_t workspace_bytes, moe_stream_t stream) {
  moe_status st = check_ff(c);
  if (st != MOE_OK) return st;
  if (c->wdtype != MOE_W_BF16) return MOE_ERR_UNSUPPORTED;
  // (of no rows dx has no address)
  if (rows < 0 || rows > kMaxRows || (rows && !dx && !dw13 && !dw2)) return MOE_ERR_INVALID_ARG;
  if (dw_dtype != MOE_BF16 && dw_dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  const bool f32 = dw_dtype == MOE_F32;
  if (accumulate && !f32) return MOE_ERR_UNSUPPORTED;
  if (!aligned16(dx) || !aligned16(dw13) || !aligned16(dw2)) return MOE_ERR_INVALID_ARG;
  const int64_t hid = c->hidden, in = c->inter, size = f32 ? 4 : 2;
  const Range r_dx = {dx, rows * hid * 2}, r_13 = {dw13, 2 * in * hid * size}, r_2 = {dw2, hid * in * size};
  if (any_overlap(r_13, {r_dx, r_2}) || any_overlap(r_dx, {r_2})) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (rows == 0) {
    cudaError_t e = cudaSuccess;
    if (!accumulate && dw13) e = launch_zero(dw13, r_13.bytes, s);
    if (!accumulate && dw2 && e == cudaSuccess) e = launch_zero(dw2, r_2.bytes, s);
    return cuda_status(e);
  }
  if (!wt || !wt->w2 || (dx && !wt->w13) || !grad || !gate_up || (dw13 && !x) || !workspace) return MOE_ERR_INVALID_ARG;
  if (!aligned16(wt->w13) || !aligned16(wt->w2) || !aligned16(grad) || !aligned16(x) || !aligned16(gate_up) || !aligned16(workspace))
    return MOE_ERR_INVALID_ARG;
  if (grad_stride < hid || grad_stride % 8 || (dw13 && (x_stride < hid || x_stride % 8))) return MOE_ERR_INVALID_ARG;
  for (const Range& o : {r_dx, r_13, r_2}) {
    if (!o.ptr) continue;
    if (rows_overlap(grad, grad_stride * 2, hid * 2, rows, o.ptr, o.bytes) ||
        (dw13 && rows_overlap(x, x_stride * 2, hid * 2, rows, o.ptr, o.bytes)) ||
        any_overlap(o, {{gate_up, rows * in * 4}, {wt->w2, hid * in * 2}, {dx ? wt->w13 : nullptr, 2 * in * hid * 2}}))
      return MOE_ERR_INVALID_ARG;
  }
  const BackwardPlan p = backward_plan(*c, rows);
  if (workspace_bytes < p.bytes) return MOE_ERR_INVALID_ARG;
  Device d;
  if (!device(&d)) return MOE_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  void *both = ws + p.both, *h = ws + p.h;
  int* status = reinterpret_cast<int*>(ws + p.status);

  // dh, and from it dg, du and h; dx; the weights' gradients in one launch
  PairLaunch one, both_w, inputs;
  for (PairLaunch* l : {&one, &both_w, &inputs}) {
    l->p.status = status;
    l->p.status_keep = l != &one;
    l->p.reduce = accumulate != 0;
  }
  one.p.M = (int)rows;
  one.p.N = c->inter;
  one.p.K = c->hidden;
  one.p.keep = dw2 != nullptr;
  const int each = exact_backward(rows, *c) ? 2 : 1;  // numbers that each of dg, du and h is the sum of
  bool ok = prepare(one, FORM_KM, each == 2 ? PAIR_DSWIGLU_LO : PAIR_DSWIGLU, {grad, grad_stride * 2, rows, hid}, {wt->w2, in * 2, hid, in}, false, d) &&
            make_map(&one.d, h, in * 2 * each, in, rows, 32, each, in * 2) &&
            make_map(&one.e, both, in * 4 * each, in, rows, 32, 2 * each, in * 2) &&
            make_map(&one.g, gate_up, in * 4, in, rows, 32, 2, in * 2);
  const Matrix up_a = {both, in * 4 * each, rows, 2 * in * each}, up_b = {x, x_stride * 2, rows, hid};
  const Matrix down_a = {grad, grad_stride * 2, rows, hid}, down_b = {h, in * 2 * each, rows, in * each};
  const int epi = f32 ? PAIR_F32 : PAIR_BF16;
  both_w.p.K = (int)rows;
  both_w.p.passes = inputs.p.passes = each;
  if (ok && dw13) {
    both_w.p.M = both_w.p.pass_a = 2 * c->inter;
    both_w.p.N = c->hidden;
    both_w.p.pass_b2 = c->inter;
    both_w.p.M2 = dw2 ? c->hidden : 0;
    both_w.p.N2 = dw2 ? c->inter : 0;
    ok = prepare(both_w, FORM_MM, epi, up_a, up_b, false, d) && prepare_out(both_w, dw13, f32) &&
         (!dw2 || prepare_second(both_w, down_a, down_b, dw2, f32));
  } else if (ok && dw2) {
    both_w.p.M = c->hidden;
    both_w.p.N = both_w.p.pass_b = c->inter;
    ok = prepare(both_w, FORM_MM, epi, down_a, down_b, false, d) && prepare_out(both_w, dw2, f32);
  }
  if (ok && dx) {
    inputs.p.M = (int)rows;
    inputs.p.N = c->hidden;
    inputs.p.K = inputs.p.pass_a = 2 * c->inter;
    ok = prepare(inputs, FORM_KM, PAIR_BF16, up_a, {wt->w13, hid * 2, 2 * in, hid}, false, d) &&
         prepare_out(inputs, dx, false);
  }
  if (!ok) return MOE_ERR_CUDA;
  cudaError_t e = launch(one, d, false, s);
  // (dx first: what it reads of dg and du is still in L2)
  if (e == cudaSuccess && dx) e = launch(inputs, d, true, s);
  if (e == cudaSuccess && (dw13 || dw2)) e = launch(both_w, d, true, s);
  return cuda_status(e);
}

}  // extern "C"
