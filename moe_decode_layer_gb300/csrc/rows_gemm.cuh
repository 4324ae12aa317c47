// Grouped matrix product of the many-row operators (tcgen05, sm_103a).
//
// Rows of x are grouped (by expert, or by adapter); group g has a weight matrix
// W_g [R, K] and the kernel computes, for each row p of the group,
//   acc[r] = sum_k W_g[r, k] x_p[k]   (+ sum_j B_a[r, j] u_p[j]  for adapters).
// The weights are the M side of the tensor-core product (128 weight rows fill the
// 128 TMEM lanes) and the rows of x the N side: with few rows per group, as in a
// wide mixture of experts, N shrinks to 16 and the kernel is a pure weight
// stream; with many it is a dense product. That is why this orientation was
// taken: padding goes to no weight byte and the accumulator columns of a row
// never mix with another row's, so a row's result does not depend on the batch.
//
// A CTA works on tiles of (2 sub-tiles of rt <= 128 weight rows) x (<= nmax rows
// of x). The two sub-tiles are the gate and the up rows of the same intermediate
// columns (EPI_SWIGLU: silu(g) * u needs no second pass) or neighbouring rows.
// rt is a run-time multiple of 8: a small matrix is cut into as many tiles as
// there are SMs; TMEM lanes past rt hold leftovers that nothing reads.
//
// Warps: 0 weight copies, 1 tensor-core issue, 2 copies of the rows of x (listed
// rows four to a copy, neighbouring ones as a box), 4..11 epilogue; the quantised
// formats add 8 warps that widen the codes into the bf16 stage. All copies are TMA
// with the 128-byte swizzle of the operands, zero-filled past K. (A first version
// gathered rows with 16-byte cp.async from four warps: with 256 rows a stage its
// loop took 5900 clocks where the tensor core needs 1024.)
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
// Arrives on bar when all earlier tcgen05.mma of this thread have completed.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// 16 accumulator columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Shared-memory operand descriptor: K-major rows of 128 bytes, 128-byte swizzle,
// 8-row groups 1024 bytes apart. addr is 1024-byte aligned (+ 32 bytes per 16 k).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)64 << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)2 << 61);
}

// Waits for a phase of an mbarrier, at most kWaitLimit probes of up to a
// microsecond each; false when the limit or another warp's (*abort) ended the wait.
// (Probes are counted: reading the global timer in this loop cost more than a stage.)
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile int* abort) {
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

struct Tile {
  int g, p0, n, rb;
};

// Rows of a launch with uniform tiles; adapters' rows are padded to 16 each.
__device__ __forceinline__ int num_rows(const GemmParams& p) {
  return p.ad_mode == AD_STEPS ? __ldg(p.adapter_off + p.num_adapters + 1) : p.rows;
}

// Tiles of one group follow one another with the row blocks of x innermost, so
// that the CTAs that read the same weights do so at the same time (L2).
__device__ __forceinline__ Tile tile_at(const GemmParams& p, int t) {
  Tile r;
  if (p.ents) {
    const int e = t / p.nrb;
    const int4 v = __ldg(p.ents + e);
    const int tb = v.w & 0xffff, ntb = v.w >> 16;
    const int local = t - (e - tb) * p.nrb;
    r.rb = local / ntb;
    const int4 u = __ldg(p.ents + (e - tb) + local % ntb);
    r.g = u.x;
    r.p0 = u.y;
    r.n = u.z;
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
  return (p.ents ? __ldg(p.nent) : (num_rows(p) + p.nmax - 1) / p.nmax) * p.nrb;
}

// The K steps of a tile: first K / 64 steps of the weights, then, for each adapter
// with rows in the tile, the steps of its rank. Every warp walks the same list. An
// adapter's rows start at multiples of 16 and its steps take the accumulator
// columns of its own rows only: what an adapter holds cannot reach another's rows.
__device__ __forceinline__ int adapter_of(const GemmParams& p, int pos) {
  int lo = 0, hi = p.num_adapters;  // largest a with off[a] <= pos (off[num_adapters] = first row without one)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(p.adapter_off + mid) <= pos) lo = mid; else hi = mid - 1;
  }
  return lo;
}
// The next adapter >= a with rows in [p0, p0 + n), or num_adapters.
__device__ __forceinline__ int adapter_next(const GemmParams& p, int a, int p0, int n) {
  while (a < p.num_adapters) {
    const int b = __ldg(p.adapter_off + a), e = __ldg(p.adapter_off + a + 1);
    if (b >= p0 + n) return p.num_adapters;
    if (e > b && e > p0) return a;
    a++;
  }
  return p.num_adapters;
}

// exp(-g) past fp32's range makes the quotient 0, as it should be.
__device__ __forceinline__ float silu_mul(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

// Widening of quantised codes to the bf16 operand.
// FP8: w = bf16(e4m3 * block scale): one rounding of the product (2^-9 relative,
// 1/32 of the codes' own step); the tensor core takes bf16 operands with the bf16
// rows of x, and a block scale of 128 k cannot be taken out of the sum over all k.
__device__ __forceinline__ uint32_t fp8x2_bf16x2(uint32_t two, float s) {
  const uint32_t h = e4m3x2_to_f16x2(two);
  const __half2 hh = *reinterpret_cast<const __half2*>(&h);
  const float2 f = __half22float2(hh);
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);
  return *reinterpret_cast<const uint32_t*>(&b);
}
// NVFP4: e2m1 * e4m3 has at most 6 significant bits: the bf16 operand is exact
// (as is the f16 product on the way: 2^-10 <= |v| <= 2688); the tensor scale
// multiplies the fp32 sum.
__device__ __forceinline__ uint32_t fp4x2_bf16x2(uint32_t byte, __half2 s) {
  const uint32_t h = e2m1x2_to_f16x2(byte);
  const float2 f = __half22float2(__hmul2(*reinterpret_cast<const __half2*>(&h), s));
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// The same with the tensor scale in the weights, where adapters share the sum:
// rounded to bf16 as the FP8 weights are.
__device__ __forceinline__ uint32_t fp4x2_bf16x2_folded(uint32_t byte, float s) {
  const uint32_t h = e2m1x2_to_f16x2(byte);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);
  return *reinterpret_cast<const uint32_t*>(&b);
}

template <int EPI, int FMT>
__global__ void __launch_bounds__(threads_of(FMT), 1)
    rows_gemm_kernel(const __grid_constant__ GemmParams p, const __grid_constant__ CUtensorMap map_w,
                     const __grid_constant__ CUtensorMap map_s, const __grid_constant__ CUtensorMap map_x,
                     const __grid_constant__ CUtensorMap map_u) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  // full, empty [kMaxStages], tmem full / empty [2], raw full / empty [kMaxRaw], drain,
  // adapter products full / empty
  __shared__ __align__(8) uint64_t s_bar[2 * kMaxStages + 4 + 2 * kMaxRaw + 3];

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
  const uint32_t ad_full = drain + 8u, ad_empty = drain + 16u;

  if (tid == 0) {
    s_abort = 0;
    // a stage is full when its weights (TMA bytes, or every widening thread and one
    // arrival in the copies' place) and its rows of x (TMA bytes) are there
    const uint32_t nfull = 1 + (FMT == FMT_BF16 ? 1 : kWidenThreads + 1);
    for (int s = 0; s < p.stages; s++) {
      mbar_init(full(s), nfull);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; b++) {
      mbar_init(tfull(b), 1);
      mbar_init(tempty(b), kEpilogueWarps);
    }
    if (FMT != FMT_BF16)
      for (int s = 0; s < p.raw_slots; s++) {
        mbar_init(rfull(s), 1);
        mbar_init(rempty(s), kWidenThreads / 32);
      }
    mbar_init(drain, 1);
    mbar_init(ad_full, kEpilogueWarps);
    mbar_init(ad_empty, kEpilogueWarps);
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
  if (p.pdl && (p.ad_mode != AD_EPILOGUE || (warp >= 4 && warp < 12))) {
    pdl_wait();
    fence_proxy_async_global();  // rows that the launch before wrote are read by TMA
  }
  pdl_launch_dependents();

  const int ntiles = num_tiles(p);
  const int main_steps = (p.K + 63) / 64;
  const int a_half = p.rt * 128;  // bytes of a sub-tile of a stage
  const uint32_t stage_bytes = p.stage_bytes;
  const bool ad_steps = p.ad_mode == AD_STEPS;
  const int per_adapter = ad_steps ? (p.rank + 63) / 64 : 0;
  // accumulator columns: [buffer][sub-tile][nmax]
  const int nbuf = 4 * p.nmax <= 512 ? 2 : 1;
  const int sub_rows = EPI == EPI_SWIGLU ? p.rt : 2 * p.rt;  // output rows per tile

  if (warp == 0) {
    // ---------------------------------------------------------------- weights
    if (lane == 0) {
      uint32_t it = 0, rit = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < ntiles; t += gridDim.x) {
        const Tile tl = tile_at(p, t);
        const bool sh = tl.g >= p.groups_main;
        const CUtensorMap* m = sh ? &map_s : &map_w;
        const int g = sh ? tl.g - p.groups_main : tl.g;
        const int y0 = tl.rb * sub_rows;
        const int y1 = EPI == EPI_SWIGLU ? y0 : y0 + p.rt, z1 = EPI == EPI_SWIGLU ? 1 : 0;
        if (FMT == FMT_BF16) {
          for (int k = 0; k < main_steps; k++, it++) {
            const int s = it % p.stages;
            if (!(ok = wait_phase(empty(s), (it / p.stages + 1) & 1, &s_abort))) break;
            const uint32_t dst = base + s * stage_bytes;
            mbar_arrive_expect_tx(full(s), 2 * a_half);
            tma_load_4d(dst, m, k * 64, y0, 0, g, full(s));
            tma_load_4d(dst + a_half, m, k * 64, y1, z1, g, full(s));
          }
        } else {
          // raw slots: 128 bytes of codes per row
          const int nraw = p.K / kmath(FMT);
          for (int k = 0; k < nraw; k++, rit++) {
            const int s = rit % p.raw_slots;
            if (!(ok = wait_phase(rempty(s), (rit / p.raw_slots + 1) & 1, &s_abort))) break;
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
            for (int k = 0; k < per_adapter; k++, it++) {
              const int s = it % p.stages;
              if (!(ok = wait_phase(empty(s), (it / p.stages + 1) & 1, &s_abort))) break;
              const uint32_t dst = base + s * stage_bytes;
              mbar_arrive_expect_tx(full(s), 2 * a_half);
              tma_load_4d(dst, &map_s, k * 64, y0, 0, a, full(s));
              tma_load_4d(dst + a_half, &map_s, k * 64, y1, z1, a, full(s));
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
    if (lane == 0) {
      uint32_t it = 0, tcount = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < ntiles; t += gridDim.x, tcount++) {
        const Tile tl = tile_at(p, t);
        const int b = tcount % nbuf;
        if (!(ok = wait_phase(tempty(b), (tcount / nbuf + 1) & 1, &s_abort))) break;
        tc_fence_after();
        // fp32 accumulators, bf16 x bf16, both K-major, M = 128
        constexpr uint32_t kDesc = (1u << 4) | (1u << 7) | (1u << 10) | (8u << 24);
        const uint32_t d0 = tmem + b * 2 * p.nmax, d1 = d0 + p.nmax;
        // one stage into the accumulators of n rows from the tile's row c on
        auto step = [&](int c, int n, bool first) {
          const int s = it % p.stages;
          if (!wait_phase(full(s), (it / p.stages) & 1, &s_abort)) return false;
          tc_fence_after();
          const uint32_t idesc = kDesc | ((uint32_t)((n + 15) >> 4) << 18);
          const uint32_t a = base + s * stage_bytes, bb = a + 2 * a_half + c * 128;
          const uint64_t da = smem_desc(a), db = smem_desc(bb), da1 = smem_desc(a + a_half);
#pragma unroll
          for (int j = 0; j < 4; j++) {
            const uint32_t acc = !first || j != 0;
            mma_bf16(d0 + c, da + 2 * j, db + 2 * j, idesc, acc);
            mma_bf16(d1 + c, da1 + 2 * j, db + 2 * j, idesc, acc);
          }
          mma_commit(empty(s));
          it++;
          return true;
        };
        for (int k = 0; ok && k < main_steps; k++) ok = step(0, tl.n, k == 0);
        if (ok && ad_steps)
          for (int a = adapter_next(p, adapter_of(p, tl.p0), tl.p0, tl.n); ok && a < p.num_adapters;
               a = adapter_next(p, a + 1, tl.p0, tl.n)) {
            const int c0 = max(__ldg(p.adapter_off + a) - tl.p0, 0);
            const int c1 = min(__ldg(p.adapter_off + a + 1) - tl.p0, tl.n);
            for (int k = 0; ok && k < per_adapter; k++) ok = step(c0, c1 - c0, false);
          }
        if (ok) mma_commit(tfull(b));
      }
      if (!ok) {
        mma_commit(drain);
        const uint64_t t0 = global_ns();
        while (!mbar_try_wait(drain, 0) && global_ns() - t0 < kDrainNs) {
        }
      }
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------------- rows of x
    uint32_t it = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < ntiles; t += gridDim.x) {
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
          for (int j = 0; j < 4; j++) v[j] = max(__ldg(p.src_row + tl.p0 + min(4 * (lane + 32 * h) + j, tl.n - 1)), 0);
          y[h] = make_int4(v[0], v[1], v[2], v[3]);
        }
      }
      const uint32_t bytes = copies * (listed ? 512u : p.box_rows * 128u);
      for (int k = 0; k < main_steps; k++, it++) {
        const int s = it % p.stages;
        if (!(ok = warp_wait(empty(s), (it / p.stages + 1) & 1, &s_abort))) break;
        if (lane == 0) mbar_arrive_expect_tx(full(s), bytes);
        __syncwarp();
        const uint32_t dst = base + s * stage_bytes + 2 * a_half;
        if (listed) {
          if (lane < copies) tma_gather4(dst + lane * 512, &map_x, k * 64, y[0], full(s));
          if (lane + 32 < copies) tma_gather4(dst + (lane + 32) * 512, &map_x, k * 64, y[1], full(s));
        } else if (lane < copies) {
          tma_load_2d(dst + lane * p.box_rows * 128, mx, k * 64, y_box + lane * p.box_rows, full(s));
        }
      }
      if (ok && ad_steps) {
        for (int a = adapter_next(p, adapter_of(p, tl.p0), tl.p0, tl.n); ok && a < p.num_adapters;
             a = adapter_next(p, a + 1, tl.p0, tl.n)) {
          const int b = max(__ldg(p.adapter_off + a) - tl.p0, 0), e = min(__ldg(p.adapter_off + a + 1) - tl.p0, tl.n);
          const int boxes = (e - b + 15) / 16;  // 16 rows each, as the adapter's are padded
          for (int k = 0; k < per_adapter; k++, it++) {
            const int s = it % p.stages;
            if (!(ok = warp_wait(empty(s), (it / p.stages + 1) & 1, &s_abort))) break;
            if (lane == 0) mbar_arrive_expect_tx(full(s), boxes * 2048u);
            __syncwarp();
            const uint32_t dst = base + s * stage_bytes + 2 * a_half + b * 128;
            if (lane < boxes) tma_load_2d(dst + lane * 2048, &map_u, k * 64, tl.p0 + b + lane * 16, full(s));
          }
        }
      }
    }
    if (!ok && lane == 0) {
      const uint64_t t0 = global_ns();
      while (global_ns() - t0 < kDrainNs) __nanosleep(1000);
    }
  } else if (warp >= 4 && warp < 12) {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3;  // this warp's 32 TMEM lanes; two warps share them, 16 columns in turn
    const int c0 = warp >= 8 ? 16 : 0;
    float* s_ad = reinterpret_cast<float*>(smem_raw + (base - smem_u32(smem_raw)) + p.ad_off);
    const int r = q * 32 + lane;
    uint32_t tcount = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < ntiles; t += gridDim.x, tcount++) {
      const Tile tl = tile_at(p, t);
      const int b = tcount % nbuf;
      if (p.ad_mode == AD_EPILOGUE) {
        // the tile's adapter products, while the tensor core works on the rest: one
        // thread per (weight row, row of x), weight rows of one sub-tile after another
        if (!(ok = warp_wait(ad_empty, (tcount + 1) & 1, &s_abort))) break;
        for (int i = tid - 128; i < tl.n * 2 * p.rt; i += 32 * kEpilogueWarps) {
          const int c = i / (2 * p.rt), wr = i % (2 * p.rt);
          const int sub = wr >= p.rt;
          const int y = tl.rb * sub_rows + (EPI == EPI_SWIGLU ? wr - sub * p.rt : wr);
          const int a = __ldg(p.ids + tl.p0 + c);
          float v = 0.0f;
          if ((unsigned)a < (unsigned)p.num_adapters && y < p.R) {
            const size_t brow = EPI == EPI_SWIGLU ? ((size_t)a * 2 + sub) * p.R + y : (size_t)a * p.R + y;
            const uint4* bp = reinterpret_cast<const uint4*>(p.b + brow * p.rank);
            const float* up = p.u32 + (size_t)(tl.p0 + c) * p.rank;
            for (int j = 0; j < p.rank / 8; j++) {
              const float4 u0 = *reinterpret_cast<const float4*>(up + 8 * j);
              const float4 u1 = *reinterpret_cast<const float4*>(up + 8 * j + 4);
              const float uu[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
              dot8_bf16_f32(v, __ldg(bp + j), uu);
            }
          }
          s_ad[i] = v;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(ad_full, 1);
        if (!(ok = warp_wait(ad_full, tcount & 1, &s_abort))) break;
      }
      if (!(ok = warp_wait(tfull(b), (tcount / nbuf) & 1, &s_abort))) break;
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
      } else if (EPI == EPI_BF16 && FMT == FMT_BF16 && p.gscale) {
        g0 = g1 = __ldg(p.gscale + tl.g);
      }
      if (q * 32 < p.rt) {
        const int y0 = tl.rb * sub_rows + r;
        const int y1 = y0 + p.rt;
        const bool ok0 = r < p.rt && y0 < p.R, ok1 = EPI != EPI_SWIGLU && r < p.rt && y1 < p.R;
        for (int c = c0; c < tl.n; c += 32) {
          // Everything that is loaded is on its way before the first sum is used, and
          // all 16 columns' results are made before the first is stored, without
          // branches: with them each column waited for the one before (225 clocks).
          uint32_t v0[16], v1[16];
          const int m = min(16, tl.n - c);
          int row_l = tl.p0 + c + (lane & 15);  // lane j: the row of out of column j
          if (p.out_row) row_l = (lane & 15) < m ? __ldg(p.out_row + row_l) : -1;
          row_l = (lane & 15) < m ? row_l : -1;
          __syncwarp();
          tmem_ld16(d0 + c, v0);
          tmem_ld16(d1 + c, v1);
          float e0[16], e1[16];
          if (EPI != EPI_SWIGLU && p.addend) {
#pragma unroll
            for (int j = 0; j < 16; j++) {
              const __nv_bfloat16* a = p.addend + (size_t)max(__shfl_sync(0xffffffffu, row_l, j), 0) * p.out_stride;
              e0[j] = __bfloat162float(a[ok0 ? y0 : 0]);
              e1[j] = __bfloat162float(a[ok1 ? y1 : 0]);
            }
          }
          if (p.ad_mode == AD_EPILOGUE) {
            const float* ad = s_ad + c * 2 * p.rt + min(r, p.rt - 1);
            const bool add = EPI != EPI_SWIGLU && p.addend;
#pragma unroll
            for (int j = 0; j < 16; j++) {
              const int at = j < m ? j * 2 * p.rt : 0;
              e0[j] = (add ? e0[j] : 0.0f) + ad[at];
              e1[j] = (add ? e1[j] : 0.0f) + ad[at + p.rt];
            }
          }
          const bool extra = p.ad_mode == AD_EPILOGUE || (EPI != EPI_SWIGLU && p.addend);
          tmem_ld_wait();
          float a0[16], a1[16];
#pragma unroll
          for (int j = 0; j < 16; j++) {
            a0[j] = __uint_as_float(v0[j]) * g0;
            a1[j] = __uint_as_float(v1[j]) * g1;
            if (extra) {
              a0[j] += e0[j];
              a1[j] += e1[j];
            }
            if (EPI == EPI_SWIGLU) a0[j] = silu_mul(a0[j], a1[j]);
          }
#pragma unroll
          for (int j = 0; j < 16; j++) {
            const int row = __shfl_sync(0xffffffffu, row_l, j);
            const size_t o = (size_t)row * p.out_stride;
            if (EPI == EPI_F32) {
              float* out = reinterpret_cast<float*>(p.out) + o;
              if (ok0 && row >= 0) out[y0] = a0[j];
              if (ok1 && row >= 0) out[y1] = a1[j];
            } else {
              __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.out) + o;
              if (ok0 && row >= 0) out[y0] = __float2bfloat16_rn(a0[j]);
              if (EPI == EPI_BF16 && ok1 && row >= 0) out[y1] = __float2bfloat16_rn(a1[j]);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(tempty(b), 1);
        if (p.ad_mode == AD_EPILOGUE) mbar_arrive(ad_empty, 1);
      }
    }
  } else if (FMT != FMT_BF16 && warp >= 12) {
    // ---------------------------------------------------------------- widening
    const int wt = tid - 384;  // 0..kWidenThreads - 1
    const int nrow = 2 * p.rt;
    uint32_t it = 0, rit = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < ntiles; t += gridDim.x) {
      const Tile tl = tile_at(p, t);
      const bool sh = tl.g >= p.groups_main;
      const int g = sh ? tl.g - p.groups_main : tl.g;
      const int y0 = tl.rb * sub_rows;
      const int nraw = p.K / kmath(FMT);
      const int parts = kmath(FMT) / 64;  // stages per raw slot
      for (int k = 0; ok && k < nraw; k++, rit++) {
        const int rs = rit % p.raw_slots;
        if (!(ok = warp_wait(rfull(rs), (rit / p.raw_slots) & 1, &s_abort))) break;
        const uint32_t raw = base + p.raw_off + rs * (2 * a_half);
        for (int h = 0; h < parts; h++, it++) {
          const int s = it % p.stages;
          if (!(ok = warp_wait(empty(s), (it / p.stages + 1) & 1, &s_abort))) break;
          const uint32_t dst = base + s * stage_bytes;
          constexpr int kChunks = FMT == FMT_FP8 ? 4 : 2;  // raw 16-byte chunks per row and stage
          for (int i = wt; i < nrow * kChunks; i += kWidenThreads) {
            const int row = i % nrow, ch = i / nrow;
            // the matrix row of this sub-tile row (scales); rows past the matrix hold zero codes
            const int sub = row >= p.rt;
            int y = y0 + (EPI == EPI_SWIGLU ? row - sub * p.rt : row);
            y = min(y, p.R - 1);
            const int yy = EPI == EPI_SWIGLU ? sub * p.R + y : y;
            const int rows_all = EPI == EPI_SWIGLU ? 2 * p.R : p.R;
            uint4 v;
            const int rc = h * kChunks + ch;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(raw + row * 128 + ((rc ^ (row & 7)) << 4)));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t o[16];
            if (FMT == FMT_FP8) {
              const float* sc = reinterpret_cast<const float*>(sh ? p.wscale_s : p.wscale);
              const float f = __ldg(sc + ((size_t)g * (rows_all / 128) + yy / 128) * (p.K / 128) + k);
#pragma unroll
              for (int j = 0; j < 4; j++) {
                o[2 * j] = fp8x2_bf16x2(w[j] & 0xffffu, f);
                o[2 * j + 1] = fp8x2_bf16x2(w[j] >> 16, f);
              }
            } else {
              const uint8_t* sc = reinterpret_cast<const uint8_t*>(sh ? p.wscale_s : p.wscale);
              const uint32_t two = __ldg(reinterpret_cast<const uint16_t*>(
                  sc + ((size_t)g * rows_all + yy) * (p.K / 16) + k * 16 + h * 4 + ch * 2));
              const uint32_t hs = e4m3x2_to_f16x2(two);
              const __half2 h2 = *reinterpret_cast<const __half2*>(&hs);
              const __half2 s0 = __low2half2(h2), s1 = __high2half2(h2);
              if (!ad_steps) {
#pragma unroll
                for (int j = 0; j < 4; j++)
#pragma unroll
                  for (int b = 0; b < 4; b++) o[4 * j + b] = fp4x2_bf16x2((w[j] >> (8 * b)) & 0xffu, j < 2 ? s0 : s1);
              } else {
                const float ts = __ldg((sh ? p.gscale_s : p.gscale) + (EPI == EPI_SWIGLU ? 2 * g + sub : g));
                const float f0 = __low2float(h2) * ts, f1 = __high2float(h2) * ts;
#pragma unroll
                for (int j = 0; j < 4; j++)
#pragma unroll
                  for (int b = 0; b < 4; b++)
                    o[4 * j + b] = fp4x2_bf16x2_folded((w[j] >> (8 * b)) & 0xffu, j < 2 ? f0 : f1);
              }
            }
            constexpr int kOut = FMT == FMT_FP8 ? 2 : 4;  // bf16 16-byte chunks written
#pragma unroll
            for (int j = 0; j < kOut; j++) {
              const int oc = ch * kOut + j;
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst + row * 128 + ((oc ^ (row & 7)) << 4)),
                           "r"(o[4 * j]), "r"(o[4 * j + 1]), "r"(o[4 * j + 2]), "r"(o[4 * j + 3])
                           : "memory");
            }
          }
          fence_proxy_async_shared();
          mbar_arrive(full(s), 1);
          if (wt == 0) mbar_arrive(full(s), 1);  // in the place of the weight copies' arrival
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(rempty(rs), 1);
      }
      // adapter steps: their weights come by TMA, loaded here; every widening thread arrives
      if (ok && ad_steps) {
        const int y1 = EPI == EPI_SWIGLU ? y0 : y0 + p.rt, z1 = EPI == EPI_SWIGLU ? 1 : 0;
        for (int a = adapter_next(p, adapter_of(p, tl.p0), tl.p0, tl.n); ok && a < p.num_adapters;
             a = adapter_next(p, a + 1, tl.p0, tl.n)) {
          for (int k = 0; k < per_adapter; k++, it++) {
            const int s = it % p.stages;
            if (!(ok = warp_wait(empty(s), (it / p.stages + 1) & 1, &s_abort))) break;
            if (wt == 0) {
              const uint32_t dst = base + s * stage_bytes;
              mbar_arrive_expect_tx(full(s), 2 * a_half);
              tma_load_4d(dst, &map_s, k * 64, y0, 0, a, full(s));
              tma_load_4d(dst + a_half, &map_s, k * 64, y1, z1, a, full(s));
            }
            mbar_arrive(full(s), 1);
          }
        }
      }
    }
    if (!ok && wt == 0) {  // as the weight warp: copies in flight land before the shared memory goes
      const uint64_t t0 = global_ns();
      while (global_ns() - t0 < kDrainNs) __nanosleep(1000);
    }
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
