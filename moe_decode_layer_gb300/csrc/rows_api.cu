// Host side of the many-row operators: checks, workspace layout, launch shapes.
// See include/moe_decode_rows.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "../../include/moe_decode_rows.h"
#include "rows_kernels.h"
#include "rows_params.h"

using namespace moe;
using namespace moe::rows;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 24;  // rows of one call
// Experts: rows handled by one round of launches; the fp32 outputs of a round's
// (row, expert) pairs are the workspace's largest part.
constexpr int64_t kRoundRows = 16384;
constexpr int kStatusKernels = 2;
constexpr int kMinN = 32;  // rows of a tile of experts' rows at least

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
// Whether the bytes at a share any with those at b.
bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const intptr_t d = static_cast<const char*>(b) - static_cast<const char*>(a);
  return a && b && d < a_bytes && -d < b_bytes;
}
// Whether rows of `width` bytes every `stride` bytes share any with those at out.
bool rows_overlap(const void* x, int64_t stride, int64_t width, int64_t rows, const void* out, int64_t bytes) {
  const intptr_t d = static_cast<const char*>(out) - static_cast<const char*>(x);
  if (d + bytes <= 0) return false;
  const int64_t last = std::min(rows - 1, (d + bytes - 1) / stride);  // the last row that starts before out's end
  return last * stride + width > d;
}
size_t up(size_t v, size_t a) { return (v + a - 1) / a * a; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static std::atomic<void*> fn{nullptr};
  void* f = fn.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      return nullptr;
    fn.store(f, std::memory_order_release);
  }
  return reinterpret_cast<EncodeTiled>(f);
}

// [groups][halves][rows][cols] row-major, copied in boxes of 128 bytes x rt rows;
// what lies past a matrix's rows or columns reads as zero.
bool make_map(CUtensorMap* m, const void* ptr, int fmt, int64_t cols, int64_t rows, int halves, int64_t groups, int rt) {
  EncodeTiled enc = encode_tiled();
  if (!enc) return false;
  const int64_t row_bytes = fmt == FMT_BF16 ? cols * 2 : fmt == FMT_FP8 ? cols : cols / 2;
  const cuuint64_t dims[4] = {(cuuint64_t)(fmt == FMT_BF16 ? cols : row_bytes), (cuuint64_t)rows, (cuuint64_t)halves,
                              (cuuint64_t)groups};
  const cuuint64_t strides[3] = {(cuuint64_t)row_bytes, (cuuint64_t)(row_bytes * rows),
                                 (cuuint64_t)(row_bytes * rows * halves)};
  const cuuint32_t box[4] = {fmt == FMT_BF16 ? 64u : 128u, (cuuint32_t)rt, 1, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return enc(m, fmt == FMT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 4,
             const_cast<void*>(ptr), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [rows][cols] bf16, row r at ptr + r * stride elements, copied 64 columns x box rows.
bool make_rows_map(CUtensorMap* m, const void* ptr, int64_t cols, int64_t rows, int64_t stride, int box) {
  EncodeTiled enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(stride * 2)};
  const cuuint32_t b[2] = {64, (cuuint32_t)box};
  const cuuint32_t one[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, b, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Device {
  int sms = 0, smem = 0, id = 0;
};
bool device(Device* d) {
  static std::atomic<uint64_t> known[64];  // per device: SMs, then shared memory; they do not change
  if (cudaGetDevice(&d->id) != cudaSuccess) return false;
  uint64_t v = d->id < 64 ? known[d->id].load(std::memory_order_relaxed) : 0;
  if (!v) {
    if (cudaDeviceGetAttribute(&d->sms, cudaDevAttrMultiProcessorCount, d->id) != cudaSuccess ||
        cudaDeviceGetAttribute(&d->smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, d->id) != cudaSuccess)
      return false;
    v = (uint64_t)d->sms << 32 | (uint32_t)d->smem;
    if (d->id < 64) known[d->id].store(v, std::memory_order_relaxed);
  }
  d->sms = (int)(v >> 32);
  d->smem = (int)(uint32_t)v;
  return d->sms <= kMaxSms;
}

// Shared memory of a launch: stages (and raw slots) for tiles of 2 rt x nmax.
struct Layout {
  int stages = 0, stage_bytes = 0, raw_off = 0, raw_slots = 0, ad_off = 0, smem = 0;
};
bool layout(int rt, int nmax, int fmt, int ksteps, int ad_mode, int smem_max, Layout* l) {
  const int a = 2 * rt * 128;
  // a quantised format's stages hold the rows of x alone, but for adapters' steps
  const bool a_smem = fmt == FMT_BF16 || ad_mode == AD_STEPS;
  l->stage_bytes = (a_smem ? a : 0) + stage_steps(fmt) * nmax * 128;
  // 1024 for alignment, 4096 for the kernel's own; the tensor core reads whole
  // 128-row sub-tiles, so up to 16 KB past a short one's start
  const int slack = 1024 + 4096 + (a_smem ? std::max(0, 128 * 128 + rt * 128 - l->stage_bytes) : 0);
  const int ad = ad_mode == AD_EPILOGUE ? nmax * 2 * rt * 4 : 0;
  int room = smem_max - slack - ad;
  l->raw_slots = 0;
  if (fmt != FMT_BF16) {
    // as many stages as tensor memory holds (2 or 3), the rest for codes
    const int most = (512 - acc_buffers(fmt, nmax) * 2 * nmax) / (64 * stage_steps(fmt));
    l->stages = std::min(most, a_smem ? (room - 2 * a) / l->stage_bytes : most);
    l->raw_slots = std::min(kMaxRaw, (room - l->stages * l->stage_bytes) / a);
    if (l->stages < 2 || l->raw_slots < 2) return false;
  } else {
    l->stages = std::min({kMaxStages, room / l->stage_bytes, std::max(ksteps, 4)});
  }
  l->raw_off = l->stages * l->stage_bytes;
  // raw slots lie behind the stages, where the reads past a short sub-tile end
  l->ad_off = l->raw_off + l->raw_slots * a;
  l->smem = l->ad_off + ad + slack - 4096;
  return l->stages >= 2;
}

// Clocks of a step with few rows of x: its waits and eight products. (200 in its place
// chooses smaller tiles and measured the same within the noise.)
constexpr double kSmallStep = 390.0;

// Rows of a sub-tile. A tile costs, per 64 k, the larger of its weight bytes (an
// SM's share of the HBM rate is about 23 bytes a clock), its operand bytes (about 55
// a clock from L2) and its tensor time (a sub-tile takes 2 n16 clocks whatever rt
// is), and its start and epilogue (45 clocks a column). The tiles go round the SMs in
// waves: rt is what makes the sum least. It is a multiple of 16 (or 8, when that
// little is wanted): a warp's results then start on a 32-byte sector. Stores of parts of
// sectors cost more than the product (8192 rows over 64 experts: 1106 us with
// rt = 104, 936 us with 128). reuse: tiles that read the same weights.
int choose_rt(int64_t R, bool swiglu, double entries, double reuse, int n, int fmt, int nmax, int ksteps, int ad_mode,
              const Device& d, double* cost_out = nullptr) {
  int best = 128;
  double least = 1e300;
  const double bytes = fmt == FMT_BF16 ? 256.0 : fmt == FMT_FP8 ? 128.0 : 72.0;
  for (int rt = 128; rt >= 8; rt -= rt > 16 ? 16 : 8) {
    Layout l;
    if (!layout(rt, nmax, fmt, ksteps, ad_mode, d.smem, &l)) continue;
    const int64_t nrb = cdiv(R, swiglu ? rt : 2 * rt);
    const double waves = std::ceil(entries * (double)nrb / d.sms);
    const double step =
        std::max({rt * bytes / (23.0 * reuse), (rt * 256.0 + n * 128.0) / 55.0, kSmallStep, 4.0 * n});
    const double cost = waves * (ksteps * step + 1500.0 + 45.0 * n);
    if (cost < least * 0.999) {
      least = cost;
      best = rt;
    }
  }
  if (cost_out) *cost_out = least;
  return best;
}

// For few rows: the CTAs that share a tile's K (1: none) and the rows of a sub-tile.
// All tiles run at once (clusters do not fill every SM: 7 of 8 are counted on); joining
// the sums costs about 1800 clocks.
int choose_split(int64_t R, bool swiglu, int entries, int nmax, int ksteps, int ad_mode, const Device& d, int* rt) {
  double least = 0.0;
  *rt = choose_rt(R, swiglu, entries, entries, nmax, FMT_BF16, nmax, ksteps, ad_mode, d, &least);
  int split = 1;
  for (int s = 2; s <= 8; s *= 2) {
    if (ksteps < 2 * s) break;
    for (int t = 128; t >= 16; t -= 16) {
      const int64_t ctas = entries * cdiv(R, swiglu ? t : 2 * t) * s;
      Layout l;
      if (ctas > d.sms * 7 / 8 || !layout(t, nmax, FMT_BF16, (int)cdiv(ksteps, s), ad_mode, d.smem, &l)) continue;
      if (l.stages * l.stage_bytes < nmax * 2 * t * 4) continue;
      const double rate = std::min(45.0, 23.0 * d.sms / ctas);
      const double cost = cdiv(ksteps, s) * std::max({t * 256.0 / rate, kSmallStep, 4.0 * nmax}) + 2500.0 + 1800.0;
      if (cost < least * 0.98) {
        least = cost;
        split = s;
        *rt = t;
      }
    }
  }
  return split;
}

struct Maps {
  CUtensorMap w, s, x, u;  // weights, the shared experts' or the adapters', rows, the rows' adapter products
};

cudaError_t launch_gemm(GemmParams& p, int epi, int fmt, Maps& m, int64_t tiles, const Layout& l, const Device& d, bool pdl, cudaStream_t st) {
  const void* k = gemm_kernel(epi, fmt);
  static std::atomic<uint64_t> ready[4][3];  // per kernel: devices whose limit is set
  if (d.id >= 64 || !(ready[epi][fmt].load() >> d.id & 1)) {
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, d.smem - 4096);
    if (e != cudaSuccess) return e;
    if (d.id < 64) ready[epi][fmt].fetch_or(1ull << d.id);
  }
  p.stages = l.stages;
  p.stage_bytes = l.stage_bytes;
  p.raw_off = l.raw_off;
  p.raw_slots = l.raw_slots;
  p.ad_off = l.ad_off;
  p.pdl = pdl;
  cudaLaunchConfig_t c = {};
  p.split = std::max(1, p.split);
  c.gridDim = dim3((unsigned)(p.split > 1 ? tiles * p.split : std::min<int64_t>(d.sms, std::max<int64_t>(tiles, 1))));
  c.blockDim = dim3(threads_of(fmt));
  // All of the SM's shared memory, used or not: a CTA takes all of its tensor memory,
  // and where CTAs of a cluster wait for one another none of them may wait for tensor
  // memory that a CTA of another cluster on its SM holds.
  c.dynamicSmemBytes = d.smem - 4096;
  c.stream = st;
  cudaLaunchAttribute a[2];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  a[1].id = cudaLaunchAttributeClusterDimension;
  a[1].val.clusterDim.x = p.split;
  a[1].val.clusterDim.y = a[1].val.clusterDim.z = 1;
  c.attrs = a;
  c.numAttrs = p.split > 1 ? 2 : 1;
  void* args[] = {&p, &m.w, &m.s, &m.x, &m.u};
  return cudaLaunchKernelExC(&c, k, args);
}

int fmt_of(int wdtype) { return wdtype == MOE_W_BF16 ? FMT_BF16 : wdtype == MOE_W_NVFP4 ? FMT_NVFP4 : FMT_FP8; }

bool widths_ok(int wdtype, int a, int b) {
  const int step = wdtype == MOE_W_BF16 ? 8 : wdtype == MOE_W_NVFP4 ? 256 : 128;
  return a % step == 0 && b % step == 0 && a <= 16384 && b <= 16384;
}

int round16(double v) { return (int)(std::ceil(v / 16.0) * 16.0); }

// ------------------------------------------------------------------ experts
struct ExpertsPlan {
  int64_t rows = 0;  // rows of a round
  int64_t positions = 0;
  int nmax = 0;
  bool spread = false;  // x is copied into the groups' order first (into y's place)
  size_t status = 0, off = 0, nent = 0, ents = 0, src_row = 0, pos = 0, h = 0, y = 0, bytes = 0;
  double touched = 0;
};
ExpertsPlan experts_plan(const moe_experts_config& c, int64_t rows) {
  ExpertsPlan p;
  p.rows = std::min(rows, kRoundRows);
  const int64_t pairs = p.rows * c.top_k;
  p.positions = pairs + p.rows * c.num_shared;
  p.touched = c.num_experts * (1.0 - std::pow(1.0 - 1.0 / c.num_experts, (double)pairs));
  // a tile holds an expert's rows unless they are far more than the average; the
  // quantised formats keep half of the shared memory for their codes
  const double avg = pairs / std::max(1.0, p.touched);
  p.nmax = std::max(kMinN, round16(2.0 * avg + 8.0));
  // Listed rows come four to a copy, about 43 clocks each: up to 128 rows a tile that
  // hides behind the weights' copies (1400 clocks a step), with 256 it is the longest
  // part (2800 clocks against the tensor core's 1024); then a pass over x pays.
  p.spread = p.nmax > 128;
  if (p.nmax > 128) p.nmax = fmt_of(c.wdtype) == FMT_BF16 ? kMaxN : 128;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at = up(at + bytes, 256);
    return o;
  };
  p.status = take((size_t)kStatusKernels * kMaxSms * 4);
  p.off = take((size_t)(c.num_experts + 1) * 4);
  p.nent = take(4);
  p.ents = take((size_t)(cdiv(pairs, kMinN) + c.num_experts + c.num_shared * cdiv(p.rows, kMinN)) * sizeof(int4));
  p.src_row = take((size_t)pairs * 4);
  p.pos = take((size_t)pairs * 4);
  p.h = take((size_t)p.positions * c.inter * 2);
  p.y = take((size_t)p.positions * c.hidden * 4);
  p.bytes = at;
  return p;
}

moe_status check_experts(const moe_experts_config* c) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (c->hidden <= 0 || c->inter <= 0 || c->num_experts <= 0 || c->top_k <= 0 || c->num_shared < 0)
    return MOE_ERR_INVALID_ARG;
  if (c->wdtype != MOE_W_BF16 && c->wdtype != MOE_W_NVFP4 && c->wdtype != MOE_W_FP8_BLOCK) return MOE_ERR_UNSUPPORTED;
  if (c->residual_dtype != MOE_BF16 && c->residual_dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (c->num_experts > 1024 || c->top_k > 16 || c->num_shared > 4 || !widths_ok(c->wdtype, c->hidden, c->inter))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// ------------------------------------------------------------------ a round of experts
struct ExpertsArgs {
  const moe_experts_config& c;
  const moe_decode_weights& wt;
  const __nv_bfloat16* x;
  int64_t x_stride;
  const int32_t* idx;
  const float* w;
  const void* residual;
  __nv_bfloat16* out;
  uint8_t* ws;
};
struct ExpertsRound {
  ExpertsPlan p;
  int64_t rows = 0, ents_max = 0;
  const __nv_bfloat16* x = nullptr;
  float* y = nullptr;
  PlanParams plan = {};
  GemmParams up = {}, down = {};
  Maps up_maps, down_maps;
  Layout up_layout, down_layout;
};

// What rows r0 .. r0 + n of a call need; nothing is launched.
moe_status prepare_round(const ExpertsArgs& a, int64_t r0, int64_t n, const Device& d, ExpertsRound* r) {
  const moe_experts_config& c = a.c;
  const moe_decode_weights& wt = a.wt;
  const int fmt = fmt_of(c.wdtype);
  const bool sh = c.num_shared > 0;
  r->rows = n;
  const ExpertsPlan& p = r->p = experts_plan(c, n);
  const int64_t pairs = n * c.top_k;
  const double blocks = std::max(1.0, std::ceil(pairs / std::max(1.0, p.touched) / p.nmax));
  const double entries = p.touched * blocks + c.num_shared * (double)cdiv(n, p.nmax);
  r->ents_max = cdiv(pairs, p.nmax) + std::min<int64_t>(c.num_experts, pairs) + c.num_shared * cdiv(n, p.nmax);
  const int n_avg = std::min<int>(p.nmax, std::max(16, round16((double)p.positions / entries)));

  PlanParams& pl = r->plan;
  pl = {};
  pl.idx = a.idx + r0 * c.top_k;
  pl.pairs = (int)pairs;
  pl.per_row = c.top_k;
  pl.groups = c.num_experts;
  pl.shared = c.num_shared;
  pl.rows = (int)n;
  pl.nmax = p.nmax;
  pl.align = 1;
  pl.off = reinterpret_cast<int*>(a.ws + p.off);
  pl.src_row = reinterpret_cast<int*>(a.ws + p.src_row);
  pl.pos = reinterpret_cast<int*>(a.ws + p.pos);
  pl.ents = reinterpret_cast<int4*>(a.ws + p.ents);
  pl.nent = reinterpret_cast<int*>(a.ws + p.nent);

  __nv_bfloat16* h = reinterpret_cast<__nv_bfloat16*>(a.ws + p.h);
  float* y = r->y = reinterpret_cast<float*>(a.ws + p.y);
  int* status = reinterpret_cast<int*>(a.ws + p.status);
  GemmParams g = {};
  g.groups_main = c.num_experts;
  g.nmax = p.nmax;
  g.ents = pl.ents;
  g.nent = pl.nent;

  // gate/up
  GemmParams& g1 = r->up = g;
  g1.R = c.inter;
  g1.K = c.hidden;
  g1.rt = choose_rt(c.inter, true, entries, blocks, n_avg, fmt, p.nmax, (c.hidden + 63) / 64, AD_NONE, d);
  g1.nrb = (int)cdiv(c.inter, g1.rt);
  g1.wscale = wt.w13_scale;
  g1.wscale_s = wt.sh_w13_scale;
  g1.gscale = wt.w13_gscale;
  g1.gscale_s = wt.sh_w13_gscale;
  g1.src_row = p.spread ? nullptr : pl.src_row;
  g1.box_rows = p.nmax % 32 ? 16 : 32;
  g1.all_rows = sh ? (int)n : 0;
  g1.all_first = (int)pairs;
  g1.out = h;
  g1.out_stride = c.inter;
  g1.status = status;
  g1.status_keep = r0 > 0;
  // down
  GemmParams& g2 = r->down = g;
  g2.R = c.hidden;
  g2.K = c.inter;
  g2.rt = choose_rt(c.hidden, false, entries, blocks, n_avg, fmt, p.nmax, (c.inter + 63) / 64, AD_NONE, d);
  g2.nrb = (int)cdiv(c.hidden, 2 * g2.rt);
  g2.wscale = wt.w2_scale;
  g2.wscale_s = wt.sh_w2_scale;
  g2.gscale = wt.w2_gscale;
  g2.gscale_s = wt.sh_w2_gscale;
  g2.box_rows = p.nmax % 32 ? 16 : 32;
  g2.out = y;
  g2.out_stride = c.hidden;
  g2.status = status + kMaxSms;
  g2.status_keep = r0 > 0;

  Maps &m1 = r->up_maps, &m2 = r->down_maps;
  const __nv_bfloat16* xr = r->x = a.x + r0 * a.x_stride;
  if (!make_map(&m1.w, wt.w13, fmt, c.hidden, c.inter, 2, c.num_experts, g1.rt) ||
      !make_map(&m2.w, wt.w2, fmt, c.inter, c.hidden, 1, c.num_experts, g2.rt) ||
      !(p.spread ? make_rows_map(&m1.x, y, c.hidden, pairs, c.hidden, g1.box_rows)
                 : make_rows_map(&m1.x, xr, c.hidden, n, a.x_stride, 1)) ||
      !make_rows_map(&m1.u, xr, c.hidden, n, a.x_stride, g1.box_rows) ||
      !make_rows_map(&m2.x, h, c.inter, p.positions, c.inter, g2.box_rows))
    return MOE_ERR_CUDA;
  m1.s = m1.w;
  m2.s = m2.u = m2.w;
  if (sh && (!make_map(&m1.s, wt.sh_w13, fmt, c.hidden, c.inter, 2, c.num_shared, g1.rt) ||
             !make_map(&m2.s, wt.sh_w2, fmt, c.inter, c.hidden, 1, c.num_shared, g2.rt)))
    return MOE_ERR_CUDA;
  if (!layout(g1.rt, p.nmax, fmt, (c.hidden + 63) / 64, AD_NONE, d.smem, &r->up_layout) ||
      !layout(g2.rt, p.nmax, fmt, (c.inter + 63) / 64, AD_NONE, d.smem, &r->down_layout))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

cudaError_t launch_round(const ExpertsArgs& a, int64_t r0, ExpertsRound& r, const Device& d, cudaStream_t s) {
  const moe_experts_config& c = a.c;
  const int fmt = fmt_of(c.wdtype);
  const int64_t pairs = r.plan.pairs;
  cudaError_t e = launch_plan(r.plan, s);
  if (e == cudaSuccess && r.p.spread)
    e = launch_spread(r.x, a.x_stride, r.plan.src_row, r.plan.off + c.num_experts, pairs, c.hidden,
                      reinterpret_cast<__nv_bfloat16*>(r.y), s);
  if (e == cudaSuccess) e = launch_gemm(r.up, EPI_SWIGLU, fmt, r.up_maps, r.ents_max * r.up.nrb, r.up_layout, d, true, s);
  if (e == cudaSuccess) e = launch_gemm(r.down, EPI_F32, fmt, r.down_maps, r.ents_max * r.down.nrb, r.down_layout, d, true, s);
  const bool f32 = c.residual_dtype == MOE_F32;
  const void* residual = a.residual ? static_cast<const uint8_t*>(a.residual) + r0 * c.hidden * (f32 ? 4 : 2) : nullptr;
  if (e == cudaSuccess)
    e = launch_combine(r.y, r.plan.pos, a.w + r0 * c.top_k, residual, f32, a.out + r0 * c.hidden, (int)r.rows, c.hidden,
                       c.top_k, c.num_shared, s);
  return e;
}

// ------------------------------------------------------------------ project
struct ProjectPlan {
  int mode = AD_NONE;
  int nmax = 0, nmax_a = 0;
  int64_t positions = 0;  // rows, with AD_STEPS those of each adapter padded to 16
  size_t status = 0, off = 0, nent = 0, ents = 0, src_row = 0, u = 0, x = 0, bytes = 0;
};
// Adapters' rows go through the tensor core, 16 columns at least for each adapter, when
// that pads not too much or there are many rows; else (decoding, where every row may
// have its own) their products are fp32 sums in the epilogue. 223 rows of 9 of 16 adapters
// (K = 320, 2 x 1168 columns, rank 64): 46 us in the epilogue, 35 as steps; 900 rows of 30
// of 64 (2048 to 4096, rank 64): 200 and 61.
constexpr int64_t kMostEpilogue = 512;
ProjectPlan project_plan(const moe_project_config& c, int64_t rows) {
  ProjectPlan p;
  const int64_t used = std::min<int64_t>(c.num_adapters, rows);
  p.mode = !c.num_adapters ? AD_NONE : rows > 64 && (rows >= 4 * used || rows >= kMostEpilogue) ? AD_STEPS : AD_EPILOGUE;
  p.positions = p.mode == AD_STEPS ? rows + 15 * used : rows;
  p.nmax = std::max(16, std::min(p.mode == AD_EPILOGUE ? 64 : kMaxN, round16((double)p.positions)));
  if (fmt_of(c.wdtype) != FMT_BF16) p.nmax = std::min(p.nmax, 128);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at = up(at + bytes, 256);
    return o;
  };
  p.status = take((size_t)kStatusKernels * kMaxSms * 4);
  if (p.mode == AD_STEPS) {
    // A x is thin: enough tiles for every SM come from the rows
    p.nmax_a = std::max(32, std::min(128, round16(rows / 140.0)));
    p.off = take((size_t)(c.num_adapters + 2) * 4);
    p.nent = take(4);
    p.ents = take((size_t)(cdiv(rows, 16) + c.num_adapters) * sizeof(int4));
    p.src_row = take((size_t)p.positions * 4);
    p.u = take((size_t)p.positions * c.rank * 4);
    p.x = take((size_t)p.positions * c.inner * 2);  // x in the adapters' order
  } else if (p.mode == AD_EPILOGUE) {
    p.u = take((size_t)rows * c.rank * 4);
  }
  p.bytes = at;
  return p;
}

moe_status check_project(const moe_project_config* c) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (c->inner <= 0 || c->outer <= 0 || c->num_adapters < 0) return MOE_ERR_INVALID_ARG;
  if (c->wdtype != MOE_W_BF16 && c->wdtype != MOE_W_NVFP4 && c->wdtype != MOE_W_FP8_BLOCK) return MOE_ERR_UNSUPPORTED;
  if (c->out_dtype != MOE_BF16 && c->out_dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (c->swiglu && c->out_dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  // (results are stored two at a time: an even number of bf16 rows will do, as a router has)
  const bool router = c->wdtype == MOE_W_BF16 && c->outer % 2 == 0;
  if (!widths_ok(c->wdtype, c->inner, router ? c->inner : c->outer) || c->outer > 16384) return MOE_ERR_UNSUPPORTED;
  if (c->num_adapters) {
    if (c->rank <= 0) return MOE_ERR_INVALID_ARG;
    if (c->num_adapters > kMaxAdapters || c->rank % 8 || c->rank > 256) return MOE_ERR_UNSUPPORTED;
  }
  return MOE_OK;
}

moe_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  cudaGetLastError();  // the error is reported here, not by a later call
  return MOE_ERR_CUDA;
}

}  // namespace

extern "C" {

moe_status moe_decode_route_check(const moe_route_config* c) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (c->num_experts <= 0 || c->top_k <= 0 || c->num_groups <= 0 || c->top_groups <= 0) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(c->scale) || c->top_groups > c->num_groups) return MOE_ERR_INVALID_ARG;
  if (c->score != MOE_ROUTE_SOFTMAX && c->score != MOE_ROUTE_SIGMOID) return MOE_ERR_UNSUPPORTED;
  if (c->logits_dtype != MOE_BF16 && c->logits_dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (c->group_best != 1 && c->group_best != 2) return MOE_ERR_UNSUPPORTED;
  if (c->num_experts > 1024 || c->top_k > 16 || c->num_groups > 32) return MOE_ERR_UNSUPPORTED;
  if (c->num_experts % c->num_groups) return MOE_ERR_UNSUPPORTED;
  if (c->top_k > c->top_groups * (c->num_experts / c->num_groups)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status moe_decode_route(const moe_route_config* c, const void* logits, int64_t stride, const float* bias,
                            int64_t rows, int32_t* idx, float* w, moe_stream_t stream) {
  const moe_status st = moe_decode_route_check(c);
  if (st != MOE_OK) return st;
  if (rows < 0 || rows > kMaxRows) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  const int align = c->logits_dtype == MOE_F32 ? 4 : 2;
  if (!logits || !idx || !w || stride < c->num_experts) return MOE_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(logits) % align || !aligned4(bias) || !aligned4(idx) || !aligned4(w))
    return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_route(*c, logits, stride, bias, rows, idx, w, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status moe_decode_experts_check(const moe_experts_config* c) { return check_experts(c); }

moe_status moe_decode_experts_workspace(const moe_experts_config* c, int64_t rows, size_t* bytes) {
  const moe_status st = check_experts(c);
  if (st != MOE_OK) return st;
  if (!bytes || rows < 0 || rows > kMaxRows) return MOE_ERR_INVALID_ARG;
  *bytes = rows ? experts_plan(*c, rows).bytes : 0;  // every part grows with the rows
  return MOE_OK;
}

moe_status moe_decode_experts(const moe_experts_config* c, const moe_decode_weights* wt, const void* x,
                              int64_t x_stride, const int32_t* idx, const float* w, const void* residual, void* out,
                              int64_t rows, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  moe_status st = check_experts(c);
  if (st != MOE_OK) return st;
  if (rows < 0 || rows > kMaxRows) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!wt || !x || !idx || !w || !out || !workspace) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(out) || !aligned16(workspace)) return MOE_ERR_INVALID_ARG;
  if (!aligned4(idx) || !aligned4(w)) return MOE_ERR_INVALID_ARG;
  if (x_stride < c->hidden || x_stride % 8) return MOE_ERR_INVALID_ARG;
  // The combine writes a round's rows after the products have read them: out may be x
  // itself, row for row, and so it may be the residual; nothing in between.
  const bool f32 = c->residual_dtype == MOE_F32;
  const int64_t out_bytes = rows * c->hidden * 2;
  if ((residual != out || f32) && overlap(residual, f32 ? 2 * out_bytes : out_bytes, out, out_bytes)) return MOE_ERR_INVALID_ARG;
  if ((x != out || (x_stride != c->hidden && rows > 1)) &&
      rows_overlap(x, x_stride * 2, c->hidden * 2, rows, out, out_bytes))
    return MOE_ERR_INVALID_ARG;
  const int fmt = fmt_of(c->wdtype);
  const bool sh = c->num_shared > 0;
  if (!wt->w13 || !wt->w2 || !aligned16(wt->w13) || !aligned16(wt->w2)) return MOE_ERR_INVALID_ARG;
  if (sh && (!wt->sh_w13 || !wt->sh_w2 || !aligned16(wt->sh_w13) || !aligned16(wt->sh_w2))) return MOE_ERR_INVALID_ARG;
  if (fmt != FMT_BF16) {
    if (!wt->w13_scale || !wt->w2_scale || (sh && (!wt->sh_w13_scale || !wt->sh_w2_scale))) return MOE_ERR_INVALID_ARG;
    if (!aligned16(wt->w13_scale) || !aligned16(wt->w2_scale) || (sh && (!aligned16(wt->sh_w13_scale) || !aligned16(wt->sh_w2_scale))))
      return MOE_ERR_INVALID_ARG;
  }
  if (fmt == FMT_NVFP4 && (!wt->w13_gscale || !wt->w2_gscale || (sh && (!wt->sh_w13_gscale || !wt->sh_w2_gscale))))
    return MOE_ERR_INVALID_ARG;
  if (fmt == FMT_NVFP4 && (!aligned4(wt->w13_gscale) || !aligned4(wt->w2_gscale) ||
                           (sh && (!aligned4(wt->sh_w13_gscale) || !aligned4(wt->sh_w2_gscale)))))
    return MOE_ERR_INVALID_ARG;
  size_t need = 0;
  moe_decode_experts_workspace(c, rows, &need);
  if (workspace_bytes < need) return MOE_ERR_INVALID_ARG;
  Device d;
  if (!device(&d)) return MOE_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const ExpertsArgs a = {*c,
                         *wt,
                         static_cast<const __nv_bfloat16*>(x),
                         x_stride,
                         idx,
                         w,
                         residual,
                         static_cast<__nv_bfloat16*>(out),
                         static_cast<uint8_t*>(workspace)};
  // The first round's and the last one's descriptors and layouts before any launch (those
  // between are the first's on other rows): what cannot be done is refused as a whole.
  const int64_t last = (rows - 1) / kRoundRows * kRoundRows;
  ExpertsRound first, end, mid;
  st = prepare_round(a, 0, std::min(rows, kRoundRows), d, &first);
  if (st == MOE_OK && last) st = prepare_round(a, last, rows - last, d, &end);
  if (st != MOE_OK) return st;
  for (int64_t r0 = 0; r0 <= last; r0 += kRoundRows) {
    ExpertsRound& r = r0 == 0 ? first : r0 == last ? end : mid;
    if (&r == &mid && (st = prepare_round(a, r0, kRoundRows, d, &mid)) != MOE_OK) return st;
    const cudaError_t e = launch_round(a, r0, r, d, s);
    if (e != cudaSuccess) return cuda_status(e);
  }
  return MOE_OK;
}

moe_status moe_decode_project_check(const moe_project_config* c) { return check_project(c); }

moe_status moe_decode_project_workspace(const moe_project_config* c, int64_t rows, size_t* bytes) {
  const moe_status st = check_project(c);
  if (st != MOE_OK) return st;
  if (!bytes || rows < 0 || rows > kMaxRows) return MOE_ERR_INVALID_ARG;
  if (rows == 0) {
    *bytes = 0;
    return MOE_OK;
  }
  // fewer rows may go the other way, whose fp32 products may need more
  const int64_t few = std::min<int64_t>({rows, kMostEpilogue - 1, std::max<int64_t>(64, 4 * (int64_t)c->num_adapters - 1)});
  const size_t status_bytes = up((size_t)kStatusKernels * kMaxSms * 4, 256);
  *bytes = std::max(project_plan(*c, rows).bytes,
                    c->num_adapters ? status_bytes + up((size_t)few * c->rank * 4, 256) : 0);
  return MOE_OK;
}

moe_status moe_decode_project(const moe_project_config* c, const moe_project_weights* wt, const void* x,
                              int64_t x_stride, const int32_t* ids, const void* addend, void* out, int64_t rows,
                              void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  moe_status st = check_project(c);
  if (st != MOE_OK) return st;
  if (rows < 0 || rows > kMaxRows) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!wt || !x || !out || !workspace || !wt->w) return MOE_ERR_INVALID_ARG;
  if (c->swiglu && addend) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(addend) || !aligned16(out) || !aligned16(workspace) || !aligned16(wt->w))
    return MOE_ERR_INVALID_ARG;
  if (x_stride < c->inner || x_stride % 8) return MOE_ERR_INVALID_ARG;
  // a tile of out is written while others still read x; its addends are read just before
  const bool f32 = c->out_dtype == MOE_F32;
  const int64_t add_bytes = rows * c->outer * 2, out_bytes = f32 ? 2 * add_bytes : add_bytes;
  if (rows_overlap(x, x_stride * 2, c->inner * 2, rows, out, out_bytes)) return MOE_ERR_INVALID_ARG;
  if ((addend != out || f32) && overlap(addend, add_bytes, out, out_bytes)) return MOE_ERR_INVALID_ARG;
  const int fmt = fmt_of(c->wdtype);
  if (fmt != FMT_BF16 && (!wt->w_scale || !aligned16(wt->w_scale))) return MOE_ERR_INVALID_ARG;
  if (fmt == FMT_NVFP4 && (!wt->w_gscale || !aligned4(wt->w_gscale))) return MOE_ERR_INVALID_ARG;
  if (c->num_adapters) {
    if (!wt->a || !wt->b || !ids || !aligned16(wt->a) || !aligned16(wt->b)) return MOE_ERR_INVALID_ARG;
    if (!aligned4(ids) || !aligned4(wt->scale)) return MOE_ERR_INVALID_ARG;
  }
  size_t need = 0;
  moe_decode_project_workspace(c, rows, &need);
  if (workspace_bytes < need) return MOE_ERR_INVALID_ARG;
  Device d;
  if (!device(&d)) return MOE_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  ProjectPlan p = project_plan(*c, rows);
  int* status = reinterpret_cast<int*>(ws + p.status);
  const bool swiglu = c->swiglu != 0;
  const int epi = swiglu ? EPI_SWIGLU : c->out_dtype == MOE_F32 ? EPI_F32 : EPI_BF16;
  const int ksteps = (c->inner + 63) / 64;

  GemmParams g = {};
  g.R = c->outer;
  g.K = c->inner;
  if (fmt == FMT_BF16 && p.nmax > 128) {
    // many rows: the tile width that fills the last round of tiles best
    double least = 1e300;
    int best = p.nmax;
    for (int n = kMaxN; n >= 96; n -= 16) {
      double cost;
      const double e = (double)cdiv(rows, n);
      choose_rt(c->outer, swiglu, e, e, n, fmt, n, ksteps, p.mode, d, &cost);
      if (cost < least * 0.995) {
        least = cost;
        best = n;
      }
    }
    p.nmax = best;
  }
  const double entries = (double)cdiv(p.positions, p.nmax);
  if (fmt == FMT_BF16 && p.mode != AD_STEPS && rows <= 64)
    g.split = choose_split(c->outer, swiglu, (int)entries, p.nmax, ksteps, p.mode, d, &g.rt);
  else
    g.rt = choose_rt(c->outer, swiglu, entries, entries, p.nmax, fmt, p.nmax, ksteps, p.mode, d);
  g.nrb = (int)cdiv(c->outer, swiglu ? g.rt : 2 * g.rt);
  g.groups_main = 1;
  g.wscale = wt->w_scale;
  g.gscale = fmt == FMT_NVFP4 ? wt->w_gscale : nullptr;
  g.box_rows = p.nmax % 32 ? 16 : 32;
  g.rows = (int)rows;
  g.nmax = p.nmax;
  g.out = out;
  g.out_stride = c->outer;
  g.addend = static_cast<const __nv_bfloat16*>(addend);
  g.status = status + kMaxSms;
  g.status_clear = p.mode == AD_STEPS ? nullptr : status;
  Maps m, ma;
  if (!make_map(&m.w, wt->w, fmt, c->inner, c->outer, swiglu ? 2 : 1, 1, g.rt) ||
      !(p.mode == AD_STEPS ? make_rows_map(&m.x, ws + p.x, c->inner, p.positions, c->inner, g.box_rows)
                           : make_rows_map(&m.x, x, c->inner, rows, x_stride, g.box_rows)))
    return MOE_ERR_CUDA;
  m.s = m.u = m.w;
  Layout l, la;
  if (!layout(g.rt, p.nmax, fmt, (int)cdiv(ksteps, std::max(1, g.split)), p.mode, d.smem, &l)) return MOE_ERR_UNSUPPORTED;

  cudaError_t e = cudaSuccess;
  g.ad_mode = p.mode;
  g.num_adapters = c->num_adapters;
  g.rank = c->rank;
  if (p.mode == AD_EPILOGUE) {
    g.ids = ids;
    g.u32 = reinterpret_cast<const float*>(ws + p.u);
    g.b = static_cast<const __nv_bfloat16*>(wt->b);
    e = launch_shrink(static_cast<const __nv_bfloat16*>(x), x_stride, static_cast<const __nv_bfloat16*>(wt->a), wt->scale, ids,
                      reinterpret_cast<float*>(ws + p.u), (int)rows, c->inner, c->rank, c->num_adapters, s);
  } else if (p.mode == AD_STEPS) {
    PlanParams pl = {};
    pl.idx = ids;
    pl.pairs = (int)rows;
    pl.per_row = 1;
    pl.groups = c->num_adapters;
    pl.rows = (int)rows;
    pl.nmax = p.nmax_a;
    pl.keep_none = 1;
    pl.align = 16;
    pl.off = reinterpret_cast<int*>(ws + p.off);
    pl.src_row = reinterpret_cast<int*>(ws + p.src_row);
    pl.ents = reinterpret_cast<int4*>(ws + p.ents);
    pl.nent = reinterpret_cast<int*>(ws + p.nent);
    // u = scale_a A_a x, as two bf16 numbers
    GemmParams ga = {};
    ga.R = c->rank;
    ga.K = c->inner;
    const double groups = std::min<double>(c->num_adapters, (double)rows);
    ga.rt = choose_rt(c->rank, false, groups * std::ceil(rows / groups / p.nmax_a), 1.0, p.nmax_a, FMT_BF16, p.nmax_a,
                      ksteps, AD_NONE, d);
    ga.nrb = (int)cdiv(c->rank, 2 * ga.rt);
    ga.groups_main = c->num_adapters;
    ga.gscale = wt->scale;
    ga.box_rows = p.nmax_a % 32 ? 16 : 32;
    ga.nmax = p.nmax_a;
    ga.ents = pl.ents;
    ga.nent = pl.nent;
    ga.out = ws + p.u;
    ga.out_stride = 2 * c->rank;
    ga.lo_off = c->rank;
    ga.status = status;
    if (!make_map(&ma.w, wt->a, FMT_BF16, c->inner, c->rank, 1, c->num_adapters, ga.rt) ||
        !make_map(&m.s, wt->b, FMT_BF16, c->rank, c->outer, swiglu ? 2 : 1, c->num_adapters, g.rt) ||
        !make_rows_map(&m.u, ws + p.u, 2 * c->rank, p.positions, 2 * c->rank, 16))
      return MOE_ERR_CUDA;
    if (!make_rows_map(&ma.x, ws + p.x, c->inner, p.positions, c->inner, ga.box_rows)) return MOE_ERR_CUDA;
    ma.s = ma.u = ma.w;
    if (!layout(ga.rt, p.nmax_a, FMT_BF16, ksteps, AD_NONE, d.smem, &la)) return MOE_ERR_UNSUPPORTED;
    const int64_t tiles = (cdiv(rows, p.nmax_a) + std::min<int64_t>(c->num_adapters, rows)) * ga.nrb;
    e = launch_plan(pl, s);
    if (e == cudaSuccess)
      e = launch_spread(static_cast<const __nv_bfloat16*>(x), x_stride, pl.src_row, pl.off + c->num_adapters + 1,
                        p.positions, c->inner, reinterpret_cast<__nv_bfloat16*>(ws + p.x), s);
    if (e == cudaSuccess) e = launch_gemm(ga, EPI_TWO, FMT_BF16, ma, tiles, la, d, true, s);
    g.adapter_off = pl.off;
    g.out_row = pl.src_row;
  }
  if (e == cudaSuccess)
    e = launch_gemm(g, epi, fmt, m, cdiv(p.positions, p.nmax) * g.nrb, l, d, p.mode != AD_NONE, s);
  return cuda_status(e);
}

moe_status moe_decode_rows_status(const void* workspace, moe_stream_t stream) {
  if (!workspace || !aligned16(workspace)) return MOE_ERR_INVALID_ARG;
  int words[kStatusKernels * kMaxSms];
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // the read-back cannot be waited for in a stream under capture, and its target is this frame
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  cudaError_t e = cudaStreamIsCapturing(s, &cap);
  if (e != cudaSuccess) return cuda_status(e);
  if (cap != cudaStreamCaptureStatusNone) return MOE_ERR_INVALID_ARG;
  Device d;
  if (!device(&d)) return MOE_ERR_CUDA;
  e = cudaMemcpyAsync(words, workspace, sizeof(words), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_status(e);
  for (int k = 0; k < kStatusKernels; k++)
    for (int i = 0; i < d.sms; i++)
      if (words[k * kMaxSms + i]) return MOE_ERR_DEVICE_TIMEOUT;
  return MOE_OK;
}

}  // extern "C"
