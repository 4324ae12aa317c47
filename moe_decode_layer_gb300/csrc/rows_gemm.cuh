// Grouped matrix product of the many-row operators (tcgen05, sm_103a).
//
// Rows of x are grouped (by expert, or by adapter); group g has a weight matrix
// W_g [R, K] and the kernel computes, for each row p of the group,
//   acc[r] = sum_k W_g[r, k] x_p[k]   (+ sum_j B_a[r, j] u_p[j]  for adapters).
// The weights are the M side of the tensor-core product (128 weight rows fill the
// 128 TMEM lanes) and the rows of x the N side: with few rows per group, as in a
// wide mixture of experts, N shrinks to 16 and the kernel is a pure weight
// stream; with many it is a dense product. That is why this orientation was
// taken: no weight byte is padding, and a row has accumulator columns of its own,
// which nothing that another row holds can reach.
//
// A CTA works on tiles of (2 sub-tiles of rt <= 128 weight rows) x (<= nmax rows
// of x). The two sub-tiles are the gate and the up rows of the same intermediate
// columns (EPI_SWIGLU: silu(g) * u needs no second pass) or neighbouring rows.
// rt is a run-time multiple of 8: a small matrix is cut into as many tiles as
// there are SMs; TMEM lanes past rt hold leftovers that nothing reads.
//
// Warps: 0 weight copies, 1 tensor-core issue, 2 copies of the rows of x (listed
// rows four to a copy, neighbouring ones as a box), 4..11 epilogue; the quantised
// formats add 8 warps that widen the codes to bf16, into tensor memory, from where the
// tensor core takes them as its A operand. (Through shared memory a step moved
// 92 to 108 KB there, 720 to 845 clocks at its 128 bytes a clock.) All copies are TMA
// with the 128-byte swizzle of the operands, zero-filled past K. (Rows gathered with
// 16-byte cp.async by four warps took 5900 clocks a step of 256 rows, where the tensor
// core needs 1024.)
//
// What bounds it: with few rows for each weight (bf16) the weights' bytes -- 1001
// rows over 512 experts of 2560 x 768, 6.07 GB, run at 6.8 to 7.0 TB/s; with many,
// the tensor core beside an epilogue that it does not overlap (256 columns of two
// sub-tiles fill tensor memory) -- 619 GFLOP of gate/up products, 8192 rows over 64
// experts of 2048 x 1024, in 439 us, 1.41 PFLOP/s. FP8 (3.0 GB for 300 rows) runs at
// 6.6 TB/s, NVFP4 (1.82 GB for 512 rows) at 2.5 TB/s: a widening warp's chain of
// waits, conversions and stores takes about 1000 clocks a step, where its bytes take 400.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "moe_params.h"
#include "ptx.cuh"
#include "rows_params.h"

namespace moe {
namespace rows {

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// Four rows of a map whose box is one row.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, int x, int4 y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc(uint32_t dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// D[tmem] (+)= A[smem] * B[smem]^T, bf16 operands, fp32 accumulators.
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// The same with A in tensor memory: lane = row, two k's a column.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Stores 32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// True in one lane of the warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t v;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(v));
  return v != 0;
}
// Arrives on bar when all earlier tcgen05.mma of this thread have completed.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// 8 accumulator columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld8(uint32_t addr, uint32_t (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(addr));
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Shared-memory operand descriptor: K-major rows of 128 bytes, 128-byte swizzle,
// 8-row groups 1024 bytes apart. addr is 1024-byte aligned (+ 32 bytes per 16 k).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)64 << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)2 << 61);
}

// All threads of the cluster's CTAs; their shared memory is in order afterwards.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// A float at this CTA's shared address in the CTA of rank r of its cluster.
__device__ __forceinline__ float ld_cluster(uint32_t addr, uint32_t r) {
  float v;
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %1, %2;\n ld.shared::cluster.f32 %0, [a];\n}\n"
      : "=f"(v)
      : "r"(addr), "r"(r)
      : "memory");
  return v;
}

// Waits for a phase of an mbarrier, at most kWaitLimit probes of up to a
// microsecond each; false when the limit or another warp's (*abort) ended the wait.
// (Probes are counted: reading the global timer in this loop cost more than a stage.)
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (mbar_test_wait(bar, parity)) return true;
  for (uint32_t i = 0; i < kWaitLimit; i++) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) == 63 && *abort) return false;
  }
  *abort = 1;
  return false;
}

// The same for a whole warp, whose lanes all get the same answer.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, wait_phase(bar, parity, abort));
}

// A place in a ring of n barriers: the slot, and the parity of its use. (Divisions
// by the number of slots took a quarter of a widening warp's step.)
struct Ring {
  uint32_t slot = 0, parity = 0;
  __device__ __forceinline__ void next(uint32_t n) {
    if (++slot == n) {
      slot = 0;
      parity ^= 1;
    }
  }
};

struct Tile {
  int g, p0, n, rb;
};

// (What the launches before this one wrote, the lists of tiles and rows among it, is read
// with plain loads behind pdl_wait(): the read-only path is for what stays as it is while
// the grid is resident, and with an early launch these do not.)

// Rows of a launch with uniform tiles; adapters' rows are padded to 16 each.
__device__ __forceinline__ int num_rows(const GemmParams& p) {
  return p.ad_mode == AD_STEPS ? p.adapter_off[p.num_adapters + 1] : p.rows;
}

// Tiles of one group follow one another with the row blocks of x innermost, so
// that the CTAs that read the same weights do so at the same time (L2).
__device__ __forceinline__ Tile tile_at(const GemmParams& p, int t) {
  Tile r;
  if (p.ents) {
    const int e = t / p.nrb;
    const int4 v = p.ents[e];
    const int tb = tile_block(v), ntb = tile_blocks(v);
    const int local = t - (e - tb) * p.nrb;
    r.rb = local / ntb;
    const int4 u = p.ents[(e - tb) + local % ntb];
    r.g = tile_group(u);
    r.p0 = tile_first(u);
    r.n = tile_rows(u);
  } else {
    const int rows = num_rows(p);
    const int ntb = (rows + p.nmax - 1) / p.nmax;
    r.rb = t / ntb;
    r.g = 0;
    r.p0 = (t % ntb) * p.nmax;
    r.n = min(p.nmax, rows - r.p0);
  }
  return r;
}
__device__ __forceinline__ int num_tiles(const GemmParams& p) {
  return (p.ents ? *p.nent : (num_rows(p) + p.nmax - 1) / p.nmax) * p.nrb;
}

// The K steps of a tile: first K / 64 steps of the weights, then, for each adapter
// with rows in the tile, the steps of its rank. Every warp walks the same list. An
// adapter's rows start at multiples of 16 and its steps take the accumulator
// columns of its own rows only: what an adapter holds cannot reach another's rows.
__device__ __forceinline__ int adapter_of(const GemmParams& p, int pos) {
  int lo = 0, hi = p.num_adapters;  // largest a with off[a] <= pos (off[num_adapters] = first row without one)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.adapter_off[mid] <= pos) lo = mid; else hi = mid - 1;
  }
  return lo;
}
// The next adapter >= a with rows in [p0, p0 + n), or num_adapters.
__device__ __forceinline__ int adapter_next(const GemmParams& p, int a, int p0, int n) {
  while (a < p.num_adapters) {
    const int b = p.adapter_off[a], e = p.adapter_off[a + 1];
    if (b >= p0 + n) return p.num_adapters;
    if (e > b && e > p0) return a;
    a++;
  }
  return p.num_adapters;
}

// CUDA's fast exp and division: at most 105 + 2 steps of fp32 (2^-16 of the value) at g = -88,
// a few near 0; the result is rounded to bf16 (2^-8) next. exp(-g) past fp32's range makes
// the quotient 0, as it should be.
__device__ __forceinline__ float silu_mul(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

// A number as hi + lo, two bf16 numbers: hi = bf16(high(v)), lo = low(v, hi). A finite one
// above bf16's largest gives that and the rest; an infinity or NaN is hi's alone, so that
// the products' sum is what the number itself would make it, and not inf - inf.
__device__ __forceinline__ float high(float v) {
  constexpr float kMost = 0x1.fep+127f;  // bf16's largest
  return fabsf(v) < INFINITY ? fminf(fmaxf(v, -kMost), kMost) : v;
}
__device__ __forceinline__ float low(float v, float hi) { return fabsf(v) < INFINITY ? v - hi : 0.0f; }

// Widening of quantised codes to the bf16 operand.
// FP8: w = bf16(e4m3 * block scale): one rounding of the product (at most 2^-8 of it,
// 1/16 of the codes' own rounding); the tensor core takes bf16 operands with the bf16
// rows of x, and a block scale of 128 k cannot be taken out of the sum over all k.
__device__ __forceinline__ uint32_t scaled_bf16x2(uint32_t f16x2, float s) {
  float2 f = __half22float2(*reinterpret_cast<const __half2*>(&f16x2));
  // both products in one instruction (FP8 479 -> 451 us, NVFP4 747 -> 703 us)
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %2};\n mul.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}\n"
      : "+f"(f.x), "+f"(f.y)
      : "f"(s));
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ void fp8x4_bf16x4(uint32_t w, float s, uint32_t& o0, uint32_t& o1) {
  uint32_t h0, h1;
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(h0), "=r"(h1)
      : "r"(w));
  o0 = scaled_bf16x2(h0, s);
  o1 = scaled_bf16x2(h1, s);
}
// Eight e2m1 codes -> eight fp16 values.
__device__ __forceinline__ void fp4x8_f16x8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// NVFP4: e2m1 * e4m3 has at most 6 significant bits: the bf16 operand is exact; the
// tensor scale multiplies the fp32 sum. (Where adapters share the sum it is
// multiplied into the weights, which are rounded to bf16 as FP8's are.)
// (Byte permutes with the codes as selectors, for all or some of the codes, were
// slower: 840 to 862 us against 803 for 512 rows at the time.)

template <int EPI, int FMT>
__global__ void __launch_bounds__(threads_of(FMT), 1)
    rows_gemm_kernel(const __grid_constant__ GemmParams p, const __grid_constant__ CUtensorMap map_w,
                     const __grid_constant__ CUtensorMap map_s, const __grid_constant__ CUtensorMap map_x,
                     const __grid_constant__ CUtensorMap map_u) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ volatile int s_in[2];  // epilogue: a tile's sums are there (odd and even tiles)
  // full, empty [kMaxStages], tmem full / empty [2], raw full / empty [kMaxRaw], drain
  __shared__ __align__(8) uint64_t s_bar[2 * kMaxStages + 4 + 2 * kMaxRaw + 1];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bar0 = smem_u32(s_bar);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  auto tfull = [&](int b) { return bar0 + 8u * (2 * kMaxStages + b); };
  auto tempty = [&](int b) { return bar0 + 8u * (2 * kMaxStages + 2 + b); };
  auto rfull = [&](int s) { return bar0 + 8u * (2 * kMaxStages + 4 + s); };
  auto rempty = [&](int s) { return bar0 + 8u * (2 * kMaxStages + 4 + kMaxRaw + s); };
  const uint32_t drain = bar0 + 8u * (2 * kMaxStages + 4 + 2 * kMaxRaw);

  if (tid == 0) {
    s_abort = 0;
    // a stage is full when its weights (TMA bytes, or every widening warp and one
    // arrival in the copies' place) and its rows of x (TMA bytes) are there
    const uint32_t nfull = 1 + (FMT == FMT_BF16 ? 1 : kWidenThreads / 32 + 1);
    for (int s = 0; s < p.stages; s++) {
      mbar_init(full(s), nfull);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; b++) {
      mbar_init(tfull(b), 1);
      mbar_init(tempty(b), epilogue_warps(FMT));
    }
    if (FMT != FMT_BF16)
      for (int s = 0; s < p.raw_slots; s++) {
        mbar_init(rfull(s), 1);
        mbar_init(rempty(s), kWidenThreads / 32);
      }
    mbar_init(drain, 1);
    mbar_init_fence();
    tma_prefetch_map(&map_w);
    tma_prefetch_map(&map_s);
    tma_prefetch_map(&map_x);
    tma_prefetch_map(&map_u);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&s_tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  // With AD_EPILOGUE the launch before this one makes u32 alone, which the epilogue
  // warps wait for; the others start on the weights and rows at once.
  if (p.pdl && (p.ad_mode != AD_EPILOGUE || (warp >= 4 && warp < 4 + epilogue_warps(FMT)))) {
    pdl_wait();
    fence_proxy_async_global();  // rows that the launch before wrote are read by TMA
  }
  pdl_launch_dependents();

  const int ntiles = num_tiles(p);
  const int main_steps = (p.K + 63) / 64;
  // Few rows: the CTAs of a cluster take parts of K of one tile, and the sums are
  // joined through distributed shared memory. (A step costs 200 to 400 clocks however
  // few rows there are: 40 of them one after another were most of a decoding
  // projection's time. 32 rows, K = 2560, 2 x 768 columns: 54 -> 46 us for a call alone.)
  const int split = FMT == FMT_BF16 ? p.split : 1;
  const int part_of = split > 1 ? blockIdx.x % split : 0;
  const int k_first = main_steps * part_of / split, k_last = main_steps * (part_of + 1) / split;
  const int t_first = split > 1 ? blockIdx.x / split : blockIdx.x;
  const int t_step = split > 1 ? ntiles : gridDim.x;
  const int a_half = p.rt * 128;  // bytes of a sub-tile of a stage
  const uint32_t stage_bytes = p.stage_bytes;
  const bool ad_steps = p.ad_mode == AD_STEPS;
  // A row's products u = A x are two bf16 numbers each, u = hi + lo, so that they
  // keep 16 bits: an adapter's steps are its rank's for hi, then again for lo.
  const int rank_steps = ad_steps ? (p.rank + 63) / 64 : 0;
  const int per_adapter = 2 * rank_steps;
  // tensor memory: accumulators [buffer][sub-tile][nmax], then the quantised formats'
  // widened weights [stage][step][sub-tile][32]
  const int nbuf = acc_buffers(FMT, p.nmax);
  const uint32_t a_tmem = tmem + nbuf * 2 * p.nmax;
  // A stage of a quantised format holds two steps, so that its waits and arrivals, some
  // 400 clocks of a widening warp's time, come half as often.
  constexpr int kHalves = stage_steps(FMT);
  const int half_bytes = p.nmax * 128;  // the rows of x of one step
  const int b_off = FMT == FMT_BF16 || ad_steps ? 2 * a_half : 0;  // the rows of x in a stage
  const int sub_rows = EPI == EPI_SWIGLU ? p.rt : 2 * p.rt;  // output rows per tile

  if (warp == 0) {
    // ---------------------------------------------------------------- weights
    if (lane == 0) {
      Ring it, rit;
      bool ok = true;
      for (int t = t_first; ok && t < ntiles; t += t_step) {
        const Tile tl = tile_at(p, t);
        const bool sh = tl.g >= p.groups_main;
        const CUtensorMap* m = sh ? &map_s : &map_w;
        const int g = sh ? tl.g - p.groups_main : tl.g;
        const int y0 = tl.rb * sub_rows;
        const int y1 = EPI == EPI_SWIGLU ? y0 : y0 + p.rt, z1 = EPI == EPI_SWIGLU ? 1 : 0;
        if (FMT == FMT_BF16) {
          for (int k = k_first; k < k_last; k++, it.next(p.stages)) {
            const uint32_t s = it.slot;
            if (!(ok = wait_phase(empty(s), it.parity ^ 1, &s_abort))) break;
            const uint32_t dst = base + s * stage_bytes;
            mbar_arrive_expect_tx(full(s), 2 * a_half);
            tma_load_4d(dst, m, k * 64, y0, 0, g, full(s));
            tma_load_4d(dst + a_half, m, k * 64, y1, z1, g, full(s));
          }
        } else {
          // raw slots: 128 bytes of codes per row
          const int nraw = p.K / kmath(FMT);
          for (int k = 0; k < nraw; k++, rit.next(p.raw_slots)) {
            const uint32_t s = rit.slot;
            if (!(ok = wait_phase(rempty(s), rit.parity ^ 1, &s_abort))) break;
            const uint32_t dst = base + p.raw_off + s * (2 * a_half);
            mbar_arrive_expect_tx(rfull(s), 2 * a_half);
            tma_load_4d(dst, m, k * 128, y0, 0, g, rfull(s));
            tma_load_4d(dst + a_half, m, k * 128, y1, z1, g, rfull(s));
          }
        }
        // (the quantised formats' adapter steps are loaded by a widening thread: a
        // parity wait on a stage is only good for who has waited for its every use)
        if (FMT == FMT_BF16 && ok && ad_steps) {
          for (int a = adapter_next(p, adapter_of(p, tl.p0), tl.p0, tl.n); ok && a < p.num_adapters;
               a = adapter_next(p, a + 1, tl.p0, tl.n)) {
            for (int k = 0; k < per_adapter; k++, it.next(p.stages)) {
              const uint32_t s = it.slot;
              if (!(ok = wait_phase(empty(s), it.parity ^ 1, &s_abort))) break;
              const uint32_t dst = base + s * stage_bytes;
              mbar_arrive_expect_tx(full(s), 2 * a_half);
              const int kx = (k < rank_steps ? k : k - rank_steps) * 64;
              tma_load_4d(dst, &map_s, kx, y0, 0, a, full(s));
              tma_load_4d(dst + a_half, &map_s, kx, y1, z1, a, full(s));
            }
          }
        }
      }
      if (!ok) {  // let the copies in flight land before the shared memory goes
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < kDrainNs) __nanosleep(1000);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- tensor core
    // The whole warp walks the loop and one lane issues: addresses and descriptors
    // stay uniform values, which the instructions take from uniform registers (a step's
    // eight products issue in 80 clocks; in a one-lane loop they took 390 to 550).
    const bool leader = elect_one();
    Ring it, acc;
    bool ok = true;
    for (int t = t_first; ok && t < ntiles; t += t_step, acc.next(nbuf)) {
      const Tile tl = tile_at(p, t);
      const int b = acc.slot;
      if (!(ok = warp_wait(tempty(b), acc.parity ^ 1, &s_abort))) break;
      tc_fence_after();
      // fp32 accumulators, bf16 x bf16, both K-major, M = 128
      constexpr uint32_t kDesc = (1u << 4) | (1u << 7) | (1u << 10) | (8u << 24);
      const uint32_t d0 = tmem + b * 2 * p.nmax, d1 = d0 + p.nmax;
      // one stage into the accumulators of n rows from the tile's row c on
      auto step = [&](int c, int n, bool first, bool main) {
        const uint32_t s = it.slot;
        if (!warp_wait(full(s), it.parity, &s_abort)) return false;
        tc_fence_after();
        const uint32_t idesc = kDesc | ((uint32_t)((n + 15) >> 4) << 18);
        const uint32_t a = base + s * stage_bytes, bb = a + b_off + c * 128;
        const uint64_t da = smem_desc(a), db = smem_desc(bb), da1 = smem_desc(a + a_half);
        if (leader) {
          if (FMT != FMT_BF16 && main) {
#pragma unroll
            for (int h = 0; h < kHalves; h++) {
              const uint32_t ta = a_tmem + (s * kHalves + h) * 64;
              const uint64_t dh = smem_desc(bb + h * half_bytes);
#pragma unroll
              for (int j = 0; j < 4; j++) {
                const uint32_t more = !first || (h | j) != 0;
                mma_bf16_ta(d0, ta + 8 * j, dh + 2 * j, idesc, more);
                mma_bf16_ta(d1, ta + 32 + 8 * j, dh + 2 * j, idesc, more);
              }
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; j++) {
              const uint32_t more = !first || j != 0;
              mma_bf16(d0 + c, da + 2 * j, db + 2 * j, idesc, more);
              mma_bf16(d1 + c, da1 + 2 * j, db + 2 * j, idesc, more);
            }
          }
          mma_commit(empty(s));
        }
        __syncwarp();
        it.next(p.stages);
        return true;
      };
      for (int k = k_first; ok && k < k_last; k += kHalves) ok = step(0, tl.n, k == k_first, true);
      if (ok && ad_steps)
        for (int a = adapter_next(p, adapter_of(p, tl.p0), tl.p0, tl.n); ok && a < p.num_adapters;
             a = adapter_next(p, a + 1, tl.p0, tl.n)) {
          const int c0 = max(p.adapter_off[a] - tl.p0, 0);
          const int c1 = min(p.adapter_off[a + 1] - tl.p0, tl.n);
          for (int k = 0; ok && k < per_adapter; k++) ok = step(c0, c1 - c0, false, false);
        }
      if (ok && leader) mma_commit(tfull(b));
    }
    if (!ok && leader) {
      mma_commit(drain);
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait(drain, 0) && global_ns() - t0 < kDrainNs) {
      }
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------------- rows of x
    Ring it;
    bool ok = true;
    for (int t = t_first; ok && t < ntiles; t += t_step) {
      const Tile tl = tile_at(p, t);
      // a group that every row belongs to has its rows in x's own order (map_u)
      const bool all = p.all_rows && tl.g >= p.groups_main;
      const bool listed = !all && p.src_row != nullptr;
      const CUtensorMap* mx = all ? &map_u : &map_x;
      const int y_box = all ? tl.p0 - p.all_first - (tl.g - p.groups_main) * p.all_rows : tl.p0;
      // listed: lane i copies rows 4 i .. 4 i + 3 and those 128 further on; the last
      // copy repeats a row, and padding takes row 0 (their columns are not read)
      int4 y[2];
      const int copies = listed ? (tl.n + 3) / 4 : (tl.n + p.box_rows - 1) / p.box_rows;
      if (listed) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
          int v[4];
#pragma unroll
          for (int j = 0; j < 4; j++) v[j] = max(p.src_row[tl.p0 + min(4 * (lane + 32 * h) + j, tl.n - 1)], 0);
          y[h] = make_int4(v[0], v[1], v[2], v[3]);
        }
      }
      const uint32_t bytes = kHalves * copies * (listed ? 512u : p.box_rows * 128u);
      for (int k = k_first; k < k_last; k += kHalves, it.next(p.stages)) {
        const uint32_t s = it.slot;
        if (!(ok = warp_wait(empty(s), it.parity ^ 1, &s_abort))) break;
        if (lane == 0) mbar_arrive_expect_tx(full(s), bytes);
        __syncwarp();
#pragma unroll
        for (int h = 0; h < kHalves; h++) {
          const uint32_t dst = base + s * stage_bytes + b_off + h * half_bytes;
          const int kx = (k + h) * 64;
          if (listed) {
            if (lane < copies) tma_gather4(dst + lane * 512, &map_x, kx, y[0], full(s));
            if (lane + 32 < copies) tma_gather4(dst + (lane + 32) * 512, &map_x, kx, y[1], full(s));
          } else if (lane < copies) {
            tma_load_2d(dst + lane * p.box_rows * 128, mx, kx, y_box + lane * p.box_rows, full(s));
          }
        }
      }
      if (ok && ad_steps) {
        for (int a = adapter_next(p, adapter_of(p, tl.p0), tl.p0, tl.n); ok && a < p.num_adapters;
             a = adapter_next(p, a + 1, tl.p0, tl.n)) {
          const int b = max(p.adapter_off[a] - tl.p0, 0), e = min(p.adapter_off[a + 1] - tl.p0, tl.n);
          const int boxes = (e - b + 15) / 16;  // 16 rows each, as the adapter's are padded
          for (int k = 0; k < per_adapter; k++, it.next(p.stages)) {
            const uint32_t s = it.slot;
            if (!(ok = warp_wait(empty(s), it.parity ^ 1, &s_abort))) break;
            if (lane == 0) mbar_arrive_expect_tx(full(s), boxes * 2048u);
            __syncwarp();
            const uint32_t dst = base + s * stage_bytes + b_off + b * 128;
            // (past hi's columns lo's follow; their weights are zeros there)
            const int kx = k < rank_steps ? k * 64 : p.rank + (k - rank_steps) * 64;
            if (lane < boxes) tma_load_2d(dst + lane * 2048, &map_u, kx, tl.p0 + b + lane * 16, full(s));
          }
        }
      }
    }
    if (!ok && lane == 0) {
      const uint64_t t0 = global_ns();
      while (global_ns() - t0 < kDrainNs) __nanosleep(1000);
    }
  } else if (warp >= 4 && warp < 4 + epilogue_warps(FMT)) {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3;  // this warp's 32 TMEM lanes; two warps share them, 8 columns in turn
    const int c0 = warp >= 8 ? 8 : 0;
    float* s_ad = reinterpret_cast<float*>(smem_raw + (base - smem_u32(smem_raw)) + p.ad_off);
    const int r = q * 32 + lane;
    Ring acc;
    uint32_t tcount = 0;
    bool ok = true;
    for (int t = t_first; ok && t < ntiles; t += t_step, tcount++, acc.next(nbuf)) {
      const Tile tl = tile_at(p, t);
      const int b = acc.slot;
      if (p.ad_mode == AD_EPILOGUE) {
        // the tile's adapter products, while the tensor core works on the rest: one
        // thread per (weight row, row of x), weight rows of one sub-tile after another
        bar_sync(1, 32 * epilogue_warps(FMT));  // the last tile's products are read
        for (int i = tid - 128; i < tl.n * 2 * p.rt; i += 32 * epilogue_warps(FMT)) {
          const int c = i / (2 * p.rt), wr = i % (2 * p.rt);
          if (split > 1 && c % split != part_of) continue;  // another CTA joins that column
          const int sub = wr >= p.rt;
          const int y = tl.rb * sub_rows + (EPI == EPI_SWIGLU ? wr - sub * p.rt : wr);
          const int a = __ldg(p.ids + tl.p0 + c);
          float v = 0.0f;
          if ((unsigned)a < (unsigned)p.num_adapters && y < p.R) {
            const size_t brow = EPI == EPI_SWIGLU ? ((size_t)a * 2 + sub) * p.R + y : (size_t)a * p.R + y;
            const uint4* bp = reinterpret_cast<const uint4*>(p.b + brow * p.rank);
            const float* up = p.u32 + (size_t)(tl.p0 + c) * p.rank;
            // four chunks' loads at a time: one by one they were most of the launch
#pragma unroll 4
            for (int j = 0; j < p.rank / 8; j++) {
              const float4 u0 = *reinterpret_cast<const float4*>(up + 8 * j);
              const float4 u1 = *reinterpret_cast<const float4*>(up + 8 * j + 4);
              const float uu[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
              dot8_bf16_f32(v, __ldg(bp + j), uu);
            }
          }
          s_ad[i] = v;
        }
      }
      if (EPI != EPI_SWIGLU && p.addend && split == 1) {  // the tile's addends on their way to L2
        const int first = tl.rb * sub_rows, cols = min(2 * p.rt, p.R - first);
        const int lines = (cols * 2 + 127) / 128 + 1;
        for (int i = tid - 128; i < tl.n * lines; i += 32 * epilogue_warps(FMT)) {
          const int pos = tl.p0 + i / lines;
          const int row = p.out_row ? p.out_row[pos] : pos;
          const int col = min(first + (i % lines) * 64, first + cols - 1);
          if (row >= 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.addend + (size_t)row * p.out_stride + col));
        }
      }
      // one warp polls, the others wait at a barrier that costs no issue slots; all
      // get the same answer and leave the loop together
      if (warp == 4) {
        const bool in = warp_wait(tfull(b), acc.parity, &s_abort);
        if (lane == 0) s_in[tcount & 1] = in;
        __syncwarp();
      }
      bar_sync(1, 32 * epilogue_warps(FMT));
      ok = s_in[tcount & 1];
      if (!ok) break;
      tc_fence_after();
      const uint32_t d0 = tmem + b * 2 * p.nmax + ((uint32_t)(q * 32) << 16), d1 = d0 + p.nmax;
      const bool sh = tl.g >= p.groups_main;
      float g0 = 1.0f, g1 = 1.0f;  // tensor scales of the two sub-tiles / the group's scale
      if (FMT == FMT_NVFP4 && !ad_steps) {
        const float* gs = sh ? p.gscale_s : p.gscale;
        const int g = sh ? tl.g - p.groups_main : tl.g;
        if (EPI == EPI_SWIGLU) {
          g0 = __ldg(gs + 2 * g);
          g1 = __ldg(gs + 2 * g + 1);
        } else {
          g0 = g1 = __ldg(gs + g);
        }
      } else if (EPI == EPI_TWO && p.gscale) {
        g0 = g1 = __ldg(p.gscale + tl.g);
      }
      if (split > 1 && q * 32 < p.rt) {
        // the partial sums, [column][weight row], where the stages were: all are used
        for (int c = c0; c < tl.n; c += 2 * epilogue_warps(FMT)) {
          uint32_t v0[8], v1[8];
          __syncwarp();
          tmem_ld8(d0 + c, v0);
          tmem_ld8(d1 + c, v1);
          tmem_ld_wait();
          const uint32_t at = base + (uint32_t)(c * 2 * p.rt + r) * 4u;
          if (r < p.rt)
#pragma unroll
            for (int j = 0; j < 8; j++)
              if (c + j < tl.n) {
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + j * 8 * p.rt), "r"(v0[j]) : "memory");
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + j * 8 * p.rt + 4 * p.rt), "r"(v1[j]) : "memory");
              }
        }
      } else if (q * 32 < p.rt) {
        const int y0 = tl.rb * sub_rows + r;
        const int y1 = y0 + p.rt;
        const bool ok0 = r < p.rt && y0 < p.R, ok1 = EPI != EPI_SWIGLU && r < p.rt && y1 < p.R;
        // Two lanes exchange a value of each pair of columns, so that a store takes two
        // neighbouring results of one column: lane 2 i those of the even column.
        const bool odd = lane & 1;
        const int yp0 = y0 & ~1, yp1 = y1 & ~1;
        // Eight columns at a time, the next eight's sums and addends on their way
        // meanwhile. No branches between columns: with them each column waited for the
        // one before (225 clocks).
        constexpr int kStep = 2 * epilogue_warps(FMT);
        const bool add = EPI != EPI_SWIGLU && p.addend;
        uint32_t n0[8], n1[8];
        __nv_bfloat16 q0[8], q1[8];
        int row_n = -1;
        auto fetch = [&](int c) {
          __syncwarp();
          tmem_ld8(d0 + c, n0);
          tmem_ld8(d1 + c, n1);
          row_n = tl.p0 + min(c + (lane & 7), tl.n - 1);  // lane j: the row of out of column j
          if (p.out_row) row_n = p.out_row[row_n];
          if (add) {
#pragma unroll
            for (int j = 0; j < 8; j++) {
              const __nv_bfloat16* a = p.addend + (size_t)max(__shfl_sync(0xffffffffu, row_n, j), 0) * p.out_stride;
              q0[j] = a[ok0 ? y0 : 0];
              q1[j] = a[ok1 ? y1 : 0];
            }
          }
        };
        if (c0 < tl.n) fetch(c0);
        for (int c = c0; c < tl.n; c += kStep) {
          float a0[8], a1[8];
          tmem_ld_wait();
          const int m = min(8, tl.n - c);
          const int row_l = row_n;
#pragma unroll
          for (int j = 0; j < 8; j++) {
            a0[j] = __uint_as_float(n0[j]);
            a1[j] = __uint_as_float(n1[j]);
            if (FMT == FMT_NVFP4 || EPI == EPI_TWO) {
              a0[j] *= g0;
              a1[j] *= g1;
            }
            if (add) {
              a0[j] += __bfloat162float(q0[j]);
              a1[j] += __bfloat162float(q1[j]);
            }
          }
          if (c + kStep < tl.n) fetch(c + kStep);
          if (p.ad_mode == AD_EPILOGUE) {
            const float* ad = s_ad + c * 2 * p.rt + min(r, p.rt - 1);
#pragma unroll
            for (int j = 0; j < 8; j++) {
              const int at = j < m ? j * 2 * p.rt : 0;
              a0[j] += ad[at];
              a1[j] += ad[at + p.rt];
            }
          }
          if (EPI == EPI_SWIGLU) {
#pragma unroll
            for (int j = 0; j < 8; j++) a0[j] = silu_mul(a0[j], a1[j]);
          }
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const int row = p.out_row ? __shfl_sync(0xffffffffu, row_l, j + odd) : tl.p0 + c + j + odd;
            const bool there = j + odd < m && row >= 0;
            const size_t o = (size_t)row * p.out_stride;
            const float x0 = __shfl_xor_sync(0xffffffffu, odd ? a0[j] : a0[j + 1], 1);
            const float2 f0 = odd ? make_float2(x0, a0[j + 1]) : make_float2(a0[j], x0);
            float2 f1 = f0;
            if (EPI != EPI_SWIGLU) {
              const float x1 = __shfl_xor_sync(0xffffffffu, odd ? a1[j] : a1[j + 1], 1);
              f1 = odd ? make_float2(x1, a1[j + 1]) : make_float2(a1[j], x1);
            }
            if (EPI == EPI_F32) {
              float* out = reinterpret_cast<float*>(p.out) + o;
              if (ok0 && there) *reinterpret_cast<float2*>(out + yp0) = f0;
              if (ok1 && there) *reinterpret_cast<float2*>(out + yp1) = f1;
            } else {
              __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.out) + o;
              constexpr bool kTwo = EPI == EPI_TWO;
              const __nv_bfloat162 h0 = kTwo ? __floats2bfloat162_rn(high(f0.x), high(f0.y)) : __floats2bfloat162_rn(f0.x, f0.y);
              const __nv_bfloat162 h1 = kTwo ? __floats2bfloat162_rn(high(f1.x), high(f1.y)) : __floats2bfloat162_rn(f1.x, f1.y);
              if (ok0 && there) *reinterpret_cast<__nv_bfloat162*>(out + yp0) = h0;
              if (EPI != EPI_SWIGLU && ok1 && there) *reinterpret_cast<__nv_bfloat162*>(out + yp1) = h1;
              if (kTwo) {  // what the rounding left
                const float2 r0 = __bfloat1622float2(h0), r1 = __bfloat1622float2(h1);
                out += p.lo_off;
                if (ok0 && there)
                  *reinterpret_cast<__nv_bfloat162*>(out + yp0) = __floats2bfloat162_rn(low(f0.x, r0.x), low(f0.y, r0.y));
                if (ok1 && there)
                  *reinterpret_cast<__nv_bfloat162*>(out + yp1) = __floats2bfloat162_rn(low(f1.x, r1.x), low(f1.y, r1.y));
              }
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(tempty(b), 1);
      }
    }
  } else if (FMT != FMT_BF16 && warp >= 4 + epilogue_warps(FMT)) {
    // ---------------------------------------------------------------- widening
    const int wt = tid - (128 + 32 * epilogue_warps(FMT));  // 0..kWidenThreads - 1
    // A thread has one row of one sub-tile, its warp's tensor-memory lane. Lanes with
    // neighbouring rows read one chunk each: the swizzle spreads them over all banks.
    const int sub = wt >> 7;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int rr = min((warp & 3) * 32 + lane, p.rt - 1);  // lanes past the sub-tile repeat its last row
    const int row = sub * p.rt + rr;
    Ring it, rit;
    bool ok = true;
    for (int t = t_first; ok && t < ntiles; t += t_step) {
      const Tile tl = tile_at(p, t);
      const bool sh = tl.g >= p.groups_main;
      const int g = sh ? tl.g - p.groups_main : tl.g;
      const int y0 = tl.rb * sub_rows;
      const int nraw = p.K / kmath(FMT);
      constexpr int kParts = kmath(FMT) / 64;          // stages per raw slot
      constexpr int kChunks = FMT == FMT_FP8 ? 4 : 2;  // 16-byte chunks of codes per row and stage
      constexpr int kOut = 32 / kChunks;               // columns made of one
      // The matrix row of this thread's sub-tile row (rows past the matrix hold zero
      // codes) and where its scales are. The scales of a slot are loaded while the
      // one before is widened.
      const int y = min(y0 + (EPI == EPI_SWIGLU ? rr : row), p.R - 1);
      const int yy = EPI == EPI_SWIGLU ? sub * p.R + y : y;
      const int rows_all = EPI == EPI_SWIGLU ? 2 * p.R : p.R;
      const float* sc8 = reinterpret_cast<const float*>(sh ? p.wscale_s : p.wscale) +
                         ((size_t)g * (rows_all / 128) + yy / 128) * (p.K / 128);
      const uint4* sc4 = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(sh ? p.wscale_s : p.wscale) +
                                                        ((size_t)g * rows_all + yy) * (p.K / 16));
      float next8 = 0.0f, ts = 1.0f;
      uint4 next4 = make_uint4(0, 0, 0, 0);
      if (FMT == FMT_FP8) next8 = __ldg(sc8); else next4 = __ldg(sc4);
      if (FMT == FMT_NVFP4 && ad_steps) ts = __ldg((sh ? p.gscale_s : p.gscale) + (EPI == EPI_SWIGLU ? 2 * g + sub : g));
      for (int k = 0; ok && k < nraw; k++, rit.next(p.raw_slots)) {
        const float f8 = next8;
        const uint32_t f4[4] = {next4.x, next4.y, next4.z, next4.w};
        if (k + 1 < nraw) {
          if (FMT == FMT_FP8) next8 = __ldg(sc8 + k + 1); else next4 = __ldg(sc4 + k + 1);
        }
        const uint32_t rs = rit.slot;
        if (!(ok = warp_wait(rfull(rs), rit.parity, &s_abort))) break;
        const uint32_t raw = base + p.raw_off + rs * (2 * a_half) + row * 128;
#pragma unroll
        for (int h = 0; h < kParts; h++) {
          const uint32_t s = it.slot;
          if (h % kHalves == 0) {
            if (!(ok = warp_wait(empty(s), it.parity ^ 1, &s_abort))) break;
            tc_fence_after();
          }
          uint4 codes[kChunks];
#pragma unroll
          for (int q = 0; q < kChunks; q++)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(codes[q].x), "=r"(codes[q].y), "=r"(codes[q].z), "=r"(codes[q].w)
                         : "r"(raw + (((h * kChunks + q) ^ (row & 7)) << 4)));
          uint32_t o[32];
#pragma unroll
          for (int q = 0; q < kChunks; q++) {
            const uint32_t w[4] = {codes[q].x, codes[q].y, codes[q].z, codes[q].w};
            if (FMT == FMT_FP8) {
#pragma unroll
              for (int j = 0; j < 4; j++)
                fp8x4_bf16x4(w[j], f8, o[(kOut * q + 2 * j) & 31], o[(kOut * q + 2 * j + 1) & 31]);
            } else {
              const uint32_t hs = e4m3x2_to_f16x2(q ? f4[h & 3] >> 16 : f4[h & 3] & 0xffffu);
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hs));
              const float f0 = ad_steps ? f.x * ts : f.x, f1 = ad_steps ? f.y * ts : f.y;
#pragma unroll
              for (int j = 0; j < 4; j++) {
                uint32_t v[4];
                fp4x8_f16x8(w[j], v);
#pragma unroll
                for (int b = 0; b < 4; b++) o[(kOut * q + 4 * j + b) & 31] = scaled_bf16x2(v[b], j < 2 ? f0 : f1);
              }
            }
          }
          tmem_st32(a_tmem + (s * kHalves + h % kHalves) * 64 + sub * 32 + lanes, o);
          if (h % kHalves == kHalves - 1) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(full(s), wt == 0 ? 2 : 1);  // thread 0: also in the weight copies' place
            it.next(p.stages);
          }
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(rempty(rs), 1);
      }
      // adapter steps: their weights come by TMA, loaded here; every widening thread arrives
      if (ok && ad_steps) {
        const int y1 = EPI == EPI_SWIGLU ? y0 : y0 + p.rt, z1 = EPI == EPI_SWIGLU ? 1 : 0;
        for (int a = adapter_next(p, adapter_of(p, tl.p0), tl.p0, tl.n); ok && a < p.num_adapters;
             a = adapter_next(p, a + 1, tl.p0, tl.n)) {
          for (int k = 0; k < per_adapter; k++, it.next(p.stages)) {
            const uint32_t s = it.slot;
            if (!(ok = warp_wait(empty(s), it.parity ^ 1, &s_abort))) break;
            if (wt == 0) {
              const uint32_t dst = base + s * stage_bytes;
              mbar_arrive_expect_tx(full(s), 2 * a_half);
              const int kx = (k < rank_steps ? k : k - rank_steps) * 64;
              tma_load_4d(dst, &map_s, kx, y0, 0, a, full(s));
              tma_load_4d(dst + a_half, &map_s, kx, y1, z1, a, full(s));
            }
            if (lane == 0) mbar_arrive(full(s), 1);
          }
        }
      }
    }
    if (!ok && wt == 0) {  // as the weight warp: copies in flight land before the shared memory goes
      const uint64_t t0 = global_ns();
      while (global_ns() - t0 < kDrainNs) __nanosleep(1000);
    }
  }

  if (split > 1) {
    // Each CTA joins every split-th column, in the order of the parts. All threads
    // come here, whatever became of their waits.
    __syncwarp();
    cluster_sync();
    if (p.pdl) pdl_wait();  // (addends may be of the launch before)
    const Tile tl = tile_at(p, min(t_first, ntiles - 1));
    const int rows_out = EPI == EPI_SWIGLU ? p.rt : 2 * p.rt;
    const int cols = (tl.n - part_of + split - 1) / split;
    const float* s_ad = reinterpret_cast<const float*>(smem_raw + (base - smem_u32(smem_raw)) + p.ad_off);
    for (int i = tid; i < cols * rows_out; i += threads_of(FMT)) {
      const int c = part_of + i / rows_out * split, wr = i % rows_out;
      const int y = tl.rb * rows_out + wr;
      if (y >= p.R) continue;
      const int at = c * 2 * p.rt + wr;
      float a0 = 0.0f, a1 = 0.0f;
      for (int k = 0; k < split; k++) {
        a0 += ld_cluster(base + at * 4u, k);
        if (EPI == EPI_SWIGLU) a1 += ld_cluster(base + (at + p.rt) * 4u, k);
      }
      if (p.ad_mode == AD_EPILOGUE) {
        a0 += s_ad[at];
        if (EPI == EPI_SWIGLU) a1 += s_ad[at + p.rt];
      }
      const size_t o = (size_t)(tl.p0 + c) * p.out_stride + y;
      if (EPI != EPI_SWIGLU && p.addend) a0 += __bfloat162float(p.addend[o]);
      if (EPI == EPI_SWIGLU) a0 = silu_mul(a0, a1);
      if (EPI == EPI_F32) reinterpret_cast<float*>(p.out)[o] = a0;
      else reinterpret_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(a0);
    }
    cluster_sync();  // no CTA leaves while another reads its sums
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
  // the status words: this CTA's, and from CTA 0 those that no CTA has
  if (tid == 0 && (s_abort || !p.status_keep)) p.status[blockIdx.x] = s_abort;
  if (blockIdx.x == 0 && !p.status_keep) {
    for (int i = gridDim.x + tid; i < kMaxSms; i += threads_of(FMT)) p.status[i] = 0;
    if (p.status_clear)
      for (int i = tid; i < kMaxSms; i += threads_of(FMT)) p.status_clear[i] = 0;
  }
}

}  // namespace rows
}  // namespace moe
