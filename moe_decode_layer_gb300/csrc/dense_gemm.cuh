// Dense matrix products of the feed-forward block and its backward pass (tcgen05, sm_103a):
// D [M, N] = A B^T over K, fp32 accumulators, bf16 or fp16 operands.
//
// Two CTAs of a cluster (a pair of SMs) work on one tile of 256 rows x bn columns with
// cta_group::2 instructions: each holds 128 rows of A and half of B's columns in shared
// memory, so that a step of 64 k moves 32 KB into each SM for 2.1 M multiplications; a CTA by
// itself would move 48 KB for a tile of 128 x 256. Both accumulators (2 x 256 columns) fill tensor
// memory: the epilogue of one tile runs beside the product of the next.
//
// The gradients contract over rows of matrices that are stored by rows, so operands come in two
// orders: k innermost (rows of x, weights of the forward pass) or the operand's own index
// innermost (W2 and W13 as the backward pass reads them, and both operands of a weight
// gradient). The tensor core takes either from a descriptor: nothing is transposed.
//
// Few tiles: the pairs of a cluster (2 or 4) take parts of K of one tile, and their sums are
// joined through distributed shared memory, in the order of the parts.
//
// int8 weights (FORM_KK8) come as codes: eight warps widen them into the stage, and the epilogue
// has four. (A pass that widened the whole matrix first cost its 3 bytes a weight: 36 us for 67
// million; 1024 rows, 4096 to 2 x 8192, 123 us with it and 89 us without.)
//
// What bounds it: with many rows the tensor core, and the power limit. 8192 rows, 4096 x 8192: the forward pass 985
// us and the backward pass 2050 us one after another, 1.68 and 1.61 PFLOP/s; the forward pass in runs of some ms 903 to 940 us
// (1.75 to 1.83). A step takes 530 clocks where its products take 512. With narrower tiles a step's copies bound it: an
// SM takes in about 64 bytes a clock from L2, so that a step of bn columns needs 256 + bn clocks
// (and the ring, 5 or 6 stages, covers a copy's latency of 2600). dh's epilogue (three results for each
// of its sums, and two inputs) runs beside the product. With few rows (the
// backward pass) the weights' bytes.
// (A warp each for A's and B's copies was slower, 562 -> 634 us for dW13; so were stages of 128 k,
// half as many, 264 -> 307 us for a backward pass of 1024 rows.)
//
// Warps: 0 copies (both CTAs), 1 tensor core (the pair's first CTA), 2 copies of codes, 4..11
// epilogue (int8: 4..7, and 8..15 widen). All copies are TMA with the operands' 128-byte swizzle;
// results leave through shared memory by TMA stores, which clip what lies past the matrix.
// Every wait is bounded; who gives up sets a flag that the others look at, and the CTA's status word.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dense_params.h"
#include "tc.cuh"

namespace moe {
namespace dense {

using namespace rows;

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// This CTA's shared address as CTA r of the cluster has it.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t r) {
  uint32_t v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(v) : "r"(addr), "r"(r));
  return v;
}
// A copy into this CTA whose bytes count on a barrier of the pair's first CTA.
__device__ __forceinline__ void tma_pair_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, int x, int y, int z, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x),
               "r"(y), "r"(z), "r"(src)
               : "memory");
}
__device__ __forceinline__ void tma_add_3d(const CUtensorMap* map, int x, int y, int z, uint32_t src) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}
__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// At most N of this thread's stores still read shared memory / are not done.
template <int N>
__device__ __forceinline__ void store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void store_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void tmem_alloc2(uint32_t dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
}
__device__ __forceinline__ void tmem_relinquish2() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
// D[tmem of both] (+)= A B^T: 256 rows, each CTA's 128 from its own shared memory.
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on bar in the CTAs of the mask when all earlier mma_pair of this thread have completed.
__device__ __forceinline__ void mma_pair_commit(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(mask)
      : "memory");
}
// Arrivals at another CTA's barrier, and waits for them. The order of what is handed over is left to fences: those of
// tcgen05 for tensor memory, and for shared memory the two below. (A release over the cluster by the arrival itself
// waits for global memory as well: 2200 clocks a tile of the epilogue, and 4096 rows, 4096 to 2 x 8192 in int8, take 797 us for 296.)
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t mapped_bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(mapped_bar) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(1000u)
      : "memory");
  return ok != 0;
}
// warp_wait for such arrivals.
__device__ __forceinline__ bool warp_wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort) {
  bool ok = false;
  for (uint32_t i = 0; !ok && i < kWaitLimit; i++) {
    ok = mbar_try_wait_cluster(bar, parity);
    if (!ok && (i & 63) == 63 && *abort) break;
  }
  if (!ok) *abort = 1;
  return __all_sync(0xffffffffu, ok);
}
// What was written to this CTA's shared memory, before an arrival; what has arrived from shared memory of the
// cluster's CTAs, after a wait. Shared memory alone.
__device__ __forceinline__ void fence_release_shared() { asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory"); }
__device__ __forceinline__ void fence_acquire_shared() { asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory"); }
// 16 accumulator columns of this thread's TMEM lane; they are there after tmem_wait16.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(addr));
}
// Waits for loads of this thread; v is one of them (as an operand, so that no use of it comes earlier).
__device__ __forceinline__ void tmem_wait16(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                 "+r"(v[15])
               :
               : "memory");
}
// The same from partial sums in shared memory, columns 512 bytes apart.
__device__ __forceinline__ void smem_ld16(uint32_t addr, uint32_t (&v)[16]) {
#pragma unroll
  for (int j = 0; j < 16; j++) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[j]) : "r"(addr + j * 512) : "memory");
}
// 16 bytes at this CTA's shared address in CTA r of the cluster.
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr, uint32_t r) {
  float4 v;
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %4, %5;\n ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n}\n"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(addr), "r"(r)
      : "memory");
  return v;
}
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* map, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(map), "r"(x), "r"(y), "r"(z) : "memory");
}

// Descriptor of an operand whose own index is innermost: blocks of 64 of it (128 bytes, 128-byte
// swizzle) x 64 k, 8 KB each, one after another; 8-k groups 1024 bytes apart. A step of 16 k is
// 2048 bytes further on.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t addr) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(8192 >> 4) << 16) | ((uint64_t)64 << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void st_shared4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 ld_shared4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
// The place of 16-byte chunk c of row r in a box of 128-byte rows, as the TMA's swizzle has it.
__device__ __forceinline__ uint32_t box_at(uint32_t box, int r, int c) { return box + r * 128 + ((c ^ (r & 7)) << 4); }

// 16 values of a row as bf16, into chunks first and first + 1 of its box.
__device__ __forceinline__ void box_bf16(uint32_t box, int r, int first, const uint32_t (&v)[16]) {
#pragma unroll
  for (int c = 0; c < 2; c++) {
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; j++) o[j] = pack_bf16(__uint_as_float(v[8 * c + 2 * j]), __uint_as_float(v[8 * c + 2 * j + 1]));
    st_shared4(box_at(box, r, first + c), o[0], o[1], o[2], o[3]);
  }
}
__device__ __forceinline__ void box_f32(uint32_t box, int r, int first, const uint32_t (&v)[16]) {
#pragma unroll
  for (int c = 0; c < 4; c++) st_shared4(box_at(box, r, first + c), v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
}

// ------------------------------------------------------------------ the kernel
struct PairTile {
  int m0, n0;
  bool second;  // of the second product
};
// Row tiles go round in groups of kGroupM, the columns outside: the pairs that run at one time
// read about as much of A as of B, and most of it from L2.
template <bool TWO>
__device__ __forceinline__ PairTile pair_tile(const PairParams& p, int t, int cols) {
  const int first = p.tiles_m * p.tiles_n;
  const bool second = TWO && t >= first;
  const int tiles_m = second ? p.tiles_m2 : p.tiles_m, tiles_n = second ? p.tiles_n2 : p.tiles_n;
  if (second) t -= first;
  const int per = kGroupM * tiles_n, group = t / per;
  const int gm = min(kGroupM, tiles_m - group * kGroupM), r = t - group * per;
  return {(group * kGroupM + r % gm) * kTileM, r / gm * cols, second};
}

template <int FORM, int EPI>
__global__ void __launch_bounds__(pair_threads(FORM), 1)
    pair_gemm_kernel(const __grid_constant__ PairParams p, const __grid_constant__ CUtensorMap map_a,
                     const __grid_constant__ CUtensorMap map_b, const __grid_constant__ CUtensorMap map_d,
                     const __grid_constant__ CUtensorMap map_e, const __grid_constant__ CUtensorMap map_g,
                     const __grid_constant__ CUtensorMap map_d2) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  // full, empty [kPairStages], tmem full / empty [2], an epilogue warp's loads [8][2], drain, codes full / empty
  __shared__ __align__(8) uint64_t s_bar[2 * kPairStages + 4 + 16 + 1 + 2 * kRawSlots];
  constexpr bool kI8 = FORM == FORM_KK8, kKK = FORM == FORM_KK || kI8;
  constexpr int kThreads = pair_threads(FORM);
  constexpr bool kTwo = FORM == FORM_MM;  // (the second product's operands are map_e and map_g)
  constexpr bool kSwiglu = EPI == PAIR_SWIGLU || EPI == PAIR_SWIGLU_F32;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bar0 = smem_u32(s_bar);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kPairStages + s); };
  auto tfull = [&](int b) { return bar0 + 8u * (2 * kPairStages + b); };
  auto tempty = [&](int b) { return bar0 + 8u * (2 * kPairStages + 2 + b); };
  auto loads = [&](int w, int i) { return bar0 + 8u * (2 * kPairStages + 4 + 2 * w + i); };
  const uint32_t drain = bar0 + 8u * (2 * kPairStages + 20);
  auto rfull = [&](int s) { return bar0 + 8u * (2 * kPairStages + 21 + s); };
  auto rempty = [&](int s) { return bar0 + 8u * (2 * kPairStages + 21 + kRawSlots + s); };
  const uint32_t crank = cluster_rank();
  const int rank = crank & 1, part = crank >> 1;
  const uint32_t first_cta = crank & ~1u;  // of the pair

  if (tid == 0) {
    s_abort = 0;
    for (int s = 0; s < p.stages; s++) {
      mbar_init(full(s), kI8 ? 1 + 8 : 1);  // copies; four widening warps of each CTA
      mbar_init(empty(s), 1);
    }
    if (kI8)
      for (int s = 0; s < p.raw_slots; s++) {
        mbar_init(rfull(s), 1);
        mbar_init(rempty(s), 4);
      }
    for (int b = 0; b < 2; b++) {
      mbar_init(tfull(b), 1);
      mbar_init(tempty(b), 2 * p.ewarps);  // the epilogue warps of both CTAs
    }
    for (int w = 0; w < 16; w++) mbar_init(loads(0, w), 1);
    mbar_init(drain, 1);
    mbar_init_fence();
    tma_prefetch_map(&map_a);
    tma_prefetch_map(&map_b);
    tma_prefetch_map(&map_d);
    tma_prefetch_map(&map_e);
  }
  if (warp == 1) {
    tmem_alloc2(smem_u32(&s_tmem), 512);
    tmem_relinquish2();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the other CTA's barriers are there
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  if (p.pdl) {
    pdl_wait();
    fence_proxy_async_global();  // what the launch before wrote is read by TMA
  }
  pdl_launch_dependents();

  const int cols = kSwiglu ? p.bn / 2 : p.bn;  // result columns of a tile
  const int ntiles = p.tiles_m * p.tiles_n + (kTwo ? p.tiles_m2 * p.tiles_n2 : 0);
  const int step = gridDim.x / (2 * p.split);
  const int t_first = blockIdx.x / (2 * p.split);
  // (codes come 128 k at a time; what lies past K is zero)
  constexpr int kCut = kI8 ? 2 : 1;
  constexpr bool kPasses = FORM == FORM_KM || FORM == FORM_MM;
  const int once = (p.K + 64 * kCut - 1) / (64 * kCut), ksteps = kPasses ? once * p.passes : once;
  const int k_first = ksteps * part / p.split * kCut, k_last = ksteps * (part + 1) / p.split * kCut;
  const int b_rows = p.bn / 2;  // of B in this CTA

  if (warp == 0) {
    // ---------------------------------------------------------------- copies
    if (lane == 0) {
      const uint32_t bars = map_rank(bar0, first_cta);  // the pair's full barriers
      Ring it;
      bool ok = true;
      // Few rows: the ring holds less of B than HBM's latency asks for; L2 takes the rest.
      auto fetch_b = [&](int n, int half, int k) {
        if (kKK) {
          tma_prefetch_3d(&map_b, k * 64, n, half);
        } else if (k < once) {
          tma_prefetch_3d(&map_b, n, k * 64, 0);
          if (b_rows > 64) tma_prefetch_3d(&map_b, n + 64, k * 64, 0);
        }
      };
      for (int t = t_first; ok && t < ntiles; t += step) {
        const PairTile tl = pair_tile<kTwo>(p, t, cols);
        const int m = tl.m0 + rank * 128;
        const int n = kSwiglu ? tl.n0 : tl.n0 + rank * b_rows, half = kSwiglu ? rank : 0;
        const CUtensorMap *ma = kTwo && tl.second ? &map_e : &map_a, *mb = kTwo && tl.second ? &map_g : &map_b;
        if (!kI8)
          for (int k = k_first; k < min(k_first + p.ahead, k_last); k++) fetch_b(n, half, k);
        // (once through K, or twice: with the second numbers of operands that are sums of two)
        for (int turn = 0; ok && turn < (kPasses ? p.passes : 1); turn++) {
          const int from = turn ? max(once, k_first) : k_first, to = kPasses && !turn && p.passes > 1 ? min(once, k_last) : k_last;
          const int x = turn * once * 64;  // K of step 0
          const int am = m + (turn && FORM == FORM_MM ? kTwo && tl.second ? p.pass_a2 : p.pass_a : 0);
          const int ax = x - (turn && FORM == FORM_KM ? p.pass_a : 0);
          const int bn = n + (turn ? kTwo && tl.second ? p.pass_b2 : p.pass_b : 0);
          for (int k = from; k < to; k++, it.next(p.stages)) {
            const uint32_t s = it.slot;
            if (!(ok = wait_phase(empty(s), it.parity ^ 1, &s_abort))) break;
            const uint32_t bar = bars + 8u * s;
            const uint32_t a = base + s * p.stage_bytes, b = a + p.a_bytes;
            if (!kI8 && p.ahead && k + p.ahead < k_last) fetch_b(n, half, k + p.ahead);
            // (the other CTA's bytes may be counted before this; the phase ends with the arrival)
            if (rank == 0) mbar_arrive_expect_tx(full(s), p.step_bytes);
            if (FORM == FORM_MM) {
              tma_pair_3d(a, ma, am, k * 64 - x, 0, bar);
              tma_pair_3d(a + 8192, ma, am + 64, k * 64 - x, 0, bar);
            } else if (rank == 0 || p.a_bytes == 128 * 128) {  // (few rows are all the first CTA's)
              tma_pair_3d(a, &map_a, k * 64 - ax, m, 0, bar);
            }
            if (FORM == FORM_KK) {
              tma_pair_3d(b, &map_b, k * 64, n, half, bar);
            } else if (!kI8) {
              tma_pair_3d(b, mb, bn, k * 64 - x, 0, bar);
              if (b_rows > 64) tma_pair_3d(b + 8192, mb, bn + 64, k * 64 - x, 0, bar);
            }
          }
        }
      }
      // every arrival that the tensor core owes this CTA's barriers
      for (int s = 0; ok && s < p.stages; s++, it.next(p.stages)) ok = wait_phase(empty(it.slot), it.parity ^ 1, &s_abort);
      if (!ok) {  // let the copies in flight land before the shared memory goes
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < kDrainNs) __nanosleep(1000);
      }
    }
  } else if (kI8 && warp == 2) {
    // ---------------------------------------------------------------- codes
    if (lane == 0) {
      Ring it;
      bool ok = true;
      for (int t = t_first; ok && t < ntiles; t += step) {
        const PairTile tl = pair_tile<kTwo>(p, t, cols);
        const int n = kSwiglu ? tl.n0 : tl.n0 + rank * b_rows, half = kSwiglu ? rank : 0;
        for (int i = 0; i < p.ahead && k_first + 2 * i < k_last; i++) tma_prefetch_3d(&map_b, (k_first + 2 * i) * 64, n, half);
        for (int k = k_first; k < k_last; k += 2, it.next(p.raw_slots)) {
          const uint32_t s = it.slot;
          if (!(ok = wait_phase(rempty(s), it.parity ^ 1, &s_abort))) break;
          if (p.ahead && k + 2 * p.ahead < k_last) tma_prefetch_3d(&map_b, (k + 2 * p.ahead) * 64, n, half);
          mbar_arrive_expect_tx(rfull(s), b_rows * 128);
          tma_load_3d(base + p.raw_off + s * (b_rows * 128), &map_b, k * 64, n, half, rfull(s));
        }
      }
      if (!ok) {
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < kDrainNs) __nanosleep(1000);
      }
    }
  } else if (kI8 && warp >= 8) {
    // ---------------------------------------------------------------- widening
    // A thread has a row of this CTA's half of B: 64 codes a step become 128 bytes of fp16, exactly, where the
    // operand's swizzle has them; the scales multiply the sums.
    // Four warps take a slot, two steps, and four the next one: a slot's waits, loads, conversions and stores take
    // about 1300 clocks of a thread and its fences more, the tensor core's two steps 1024. (An even number of slots: each
    // slot is one group's, which so waits for its every use. Steps are released in order, and a group has waited
    // for a later one than the stage's use before last: three stages at least.)
    const int row = (warp & 3) * 32 + lane, group = (warp - 8) >> 2;
    const uint32_t bars = map_rank(bar0, first_cta);
    const bool mine = row < b_rows;
    Ring it, rit;
    uint32_t turn = 0;
    bool ok = true;
    for (int t = t_first; ok && t < ntiles; t += step) {
      for (int k = k_first; ok && k < k_last; k += 2, rit.next(p.raw_slots)) {
        if ((turn++ & 1) != group) {
          it.next(p.stages);
          it.next(p.stages);
          continue;
        }
        const uint32_t rs = rit.slot, raw = base + p.raw_off + rs * (b_rows * 128) + row * 128;
        if (!(ok = warp_wait(rfull(rs), rit.parity, &s_abort))) break;
        uint32_t o[2][32];
        if (mine) {
#pragma unroll
          for (int h = 0; h < 2; h++)
#pragma unroll
            for (int c = 0; c < 4; c++) {
              const uint4 q = ld_shared4(raw + (((h * 4 + c) ^ (row & 7)) << 4));
              const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
              for (int j = 0; j < 4; j++) int8x4_f16x4(w[j], o[h][8 * c + 2 * j], o[h][8 * c + 2 * j + 1]);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(rempty(rs), 1);
        // (Both steps are told at once, behind one pair of fences. The second's stage does not wait for the first's product.)
        uint32_t told[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const uint32_t s = it.slot, to = base + s * p.stage_bytes + p.a_bytes + row * 128;
          if (!(ok = ok && warp_wait(empty(s), it.parity ^ 1, &s_abort))) break;
          if (mine) {
#pragma unroll
            for (int c = 0; c < 8; c++)
              st_shared4(to + ((c ^ (row & 7)) << 4), o[h][4 * c], o[h][4 * c + 1], o[h][4 * c + 2], o[h][4 * c + 3]);
          }
          told[h] = bars + 8u * s;
          it.next(p.stages);
        }
        if (!ok) break;
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
          fence_release_shared();
          mbar_arrive_cluster(told[0]);
          mbar_arrive_cluster(told[1]);
        }
      }
    }
  } else if (warp == 1 && rank == 0) {
    // ---------------------------------------------------------------- tensor core
    const bool leader = elect_one();
    const uint16_t both = (uint16_t)(3u << first_cta);
    Ring it, acc;
    bool ok = true;
    for (int t = t_first; ok && t < ntiles; t += step, acc.next(2)) {
      const int b = acc.slot;
      if (!(ok = warp_wait_cluster(tempty(b), acc.parity ^ 1, &s_abort))) break;
      tc_fence_after();
      const uint32_t d = tmem + b * 256;
      for (int k = k_first; k < k_last; k++, it.next(p.stages)) {
        const uint32_t s = it.slot;
        if (!(ok = kI8 ? warp_wait_cluster(full(s), it.parity, &s_abort) : warp_wait(full(s), it.parity, &s_abort))) break;
        if (kI8) fence_acquire_shared();
        tc_fence_after();
        const uint32_t at = base + s * p.stage_bytes;
        const uint64_t da = FORM == FORM_MM ? smem_desc_mn(at) : smem_desc(at);
        const uint64_t db = kKK ? smem_desc(at + p.a_bytes) : smem_desc_mn(at + p.a_bytes);
        constexpr int kA = FORM == FORM_MM ? 2048 >> 4 : 2, kB = kKK ? 2 : 2048 >> 4;
        if (leader) {
#pragma unroll
          for (int j = 0; j < 4; j++) mma_pair(d, da + kA * j, db + kB * j, p.idesc, k != k_first || j != 0);
          mma_pair_commit(empty(s), both);
        }
        __syncwarp();
      }
      if (ok && leader) mma_pair_commit(tfull(b), both);
    }
    if (!ok && leader) {
      mma_pair_commit(drain, (uint16_t)(1u << crank));
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait(drain, 0) && global_ns() - t0 < kDrainNs) {
      }
    }
  }

  // ------------------------------------------------------------------ epilogue
  const int ew = warp - 4;
  const uint32_t boxes = base + p.box_off + max(ew, 0) * p.bufs * kStageBox;
  bool ok = true;
  // Columns of a box: a row of it is 128 bytes.
  constexpr int kBox = EPI == PAIR_F32 || EPI == PAIR_SWIGLU_F32 ? 32 : 64;
  constexpr bool kLo = EPI == PAIR_DSWIGLU_LO, kGrad = EPI == PAIR_DSWIGLU || kLo;
  constexpr bool kThree = EPI == PAIR_SWIGLU || kGrad;  // three boxes at once, else two in turn
  constexpr bool kTurns = !kThree && !kI8;  // (int8: one box, and another stage)
  const int nbox = cols / kBox;
  const bool asks = kGrad || (EPI == PAIR_BF16 && p.addend);  // a unit's inputs come by TMA
  uint32_t asked = 0, landed = 0, units = 0;
  auto there = [&](const PairTile& tl, int box, int q) {
    const bool two = kTwo && tl.second;
    return tl.m0 + rank * 128 + q * 32 < (two ? p.M2 : p.M) && tl.n0 + box * kBox < (two ? p.N2 : p.N);
  };
  // int8: the scales of this lane's row, and of a tile's columns, in shared memory (each warp's own): on their
  // way while the sums are made. (Loaded where they are used, they took 8 us of a tile's epilogue.)
  const uint32_t scales = base + p.scale_off + max(ew, 0) * 1024;
  auto row_scale = [&](const PairTile& tl, int q) {
    return kI8 ? p.row_scale[min(tl.m0 + rank * 128 + q * 32 + lane, p.M - 1)] : 1.0f;
  };
  auto column_scales = [&](const PairTile& tl) {
    if constexpr (kI8) {
      __syncwarp();
#pragma unroll 4
      for (int c = lane; c < p.bn; c += 32) {
        const int half = kSwiglu && c >= p.bn / 2, n = tl.n0 + c - half * (p.bn / 2);  // (past N: the last one's, not used)
        const float v = __ldg(p.col_scale + half * p.N + min(n, p.N - 1));
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(scales + c * 4), "f"(v) : "memory");
      }
      __syncwarp();
    }
  };
  // Asks for the next unit's inputs into its boxes, which the store before the last one has left.
  auto ask = [&](const PairTile& tl, int box, int q) {
    const uint32_t i = asked++, bar = loads(ew, i & 1);
    if (lane == 0) {
      const int row = tl.m0 + rank * 128 + q * 32, col = tl.n0 + box * 64;
      store_wait_read<0>();
      if (kGrad) {
        mbar_arrive_expect_tx(bar, 2 * kStageBox);
        tma_load_3d(boxes, &map_g, col, row, 0, bar);
        tma_load_3d(boxes + kStageBox, &map_g, col, row, 1, bar);
      } else {
        mbar_arrive_expect_tx(bar, kStageBox);
        tma_load_3d(boxes + (kTurns ? i & 1 : 0) * kStageBox, &map_g, col, row, 0, bar);
      }
    }
    __syncwarp();
  };
  // One box: 32 rows of the quadrant q. get(c, v): accumulator columns c .. c + 15 of this lane's row, there
  // after wait(v).
  auto unit = [&](const PairTile& tl, int box, int q, float rs, auto get, auto wait) {
    const int row0 = tl.m0 + rank * 128 + q * 32, col0 = tl.n0 + box * kBox;
    const int row = min(row0 + lane, p.M - 1);
    const uint32_t n = units++, at = kTurns ? boxes + (n & 1) * kStageBox : boxes;
    auto scaled = [&](uint32_t (&v)[16], int c) {  // accumulator columns c .. c + 15
      if constexpr (kI8) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const uint4 w = ld_shared4(scales + (c + 4 * j) * 4);
          const uint32_t f[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int i = 0; i < 4; i++) v[4 * j + i] = __float_as_uint(__uint_as_float(v[4 * j + i]) * (rs * __uint_as_float(f[i])));
        }
      }
    };
    if (asks) {
      ok = ok && warp_wait(loads(ew, n & 1), (n >> 1) & 1, &s_abort);
      if (!ok) return;
      landed++;
    } else {
      if (lane == 0) {
        if (kTurns) store_wait_read<1>();
        else store_wait_read<0>();
      }
      __syncwarp();
    }
    // (16 columns at a time, not unrolled: a launch's first tile waits for its code, and unrolled over
    // 32 columns, several thousand instructions, that took 3 us)
#pragma unroll 1
    for (int h = 0; h < kBox / 16; h++) {
      const int c0 = col0 + h * 16;
      uint32_t v[16];
      get(box * kBox + h * 16, v);
      if (EPI == PAIR_SWIGLU || EPI == PAIR_SWIGLU_F32) {
        uint32_t u[16];
        get(p.bn / 2 + box * kBox + h * 16, u);
        wait(v);
        wait(u);
        scaled(v, box * kBox + h * 16);
        scaled(u, p.bn / 2 + box * kBox + h * 16);
        if (EPI == PAIR_SWIGLU && p.keep) {
          box_bf16(at + kStageBox, lane, 2 * h, v);
          box_bf16(at + 2 * kStageBox, lane, 2 * h, u);
        }
#pragma unroll
        for (int j = 0; j < 16; j++) {
          const float a = __uint_as_float(v[j]), b = __uint_as_float(u[j]);
          v[j] = __float_as_uint(EPI == PAIR_SWIGLU ? silu_mul(a, b) : silu_mul_f32(a, b));
        }
      } else {
        wait(v);
      }
      if (kGrad) {
#pragma unroll
        for (int c = 0; c < 2; c++) {
          const uint32_t ag = box_at(at, lane, 2 * h + c), au = ag + kStageBox;
          const uint4 g4 = ld_shared4(ag), u4 = ld_shared4(au);
          const uint32_t gw[4] = {g4.x, g4.y, g4.z, g4.w}, uw[4] = {u4.x, u4.y, u4.z, u4.w};
          uint32_t dg[4], du[4], hh[4], l[3][4];
#pragma unroll
          for (int j = 0; j < 4; j++) {
            float a[2], b[2], w[2];
#pragma unroll
            for (int e = 0; e < 2; e++) {
              const float g = e ? bf16hi(gw[j]) : bf16lo(gw[j]), u = e ? bf16hi(uw[j]) : bf16lo(uw[j]);
              const float dh = __uint_as_float(v[8 * c + 2 * j + e]);
              const float sig = __fdividef(1.0f, 1.0f + __expf(-g)), s = g * sig;
              w[e] = s * u;
              b[e] = dh * s;
              a[e] = dh * u * (sig + s * (1.0f - sig));
            }
            if (kLo) {
              dg[j] = pack_bf16(high(a[0]), high(a[1]));
              du[j] = pack_bf16(high(b[0]), high(b[1]));
              hh[j] = pack_bf16(high(w[0]), high(w[1]));
              l[0][j] = pack_bf16(low(a[0], bf16lo(dg[j])), low(a[1], bf16hi(dg[j])));
              l[1][j] = pack_bf16(low(b[0], bf16lo(du[j])), low(b[1], bf16hi(du[j])));
              l[2][j] = pack_bf16(low(w[0], bf16lo(hh[j])), low(w[1], bf16hi(hh[j])));
            } else {
              dg[j] = pack_bf16(a[0], a[1]);
              du[j] = pack_bf16(b[0], b[1]);
              hh[j] = pack_bf16(w[0], w[1]);
            }
          }
          st_shared4(ag, dg[0], dg[1], dg[2], dg[3]);
          st_shared4(au, du[0], du[1], du[2], du[3]);
          st_shared4(ag + 2 * kStageBox, hh[0], hh[1], hh[2], hh[3]);
          if (kLo)
#pragma unroll
            for (int i = 0; i < 3; i++) st_shared4(ag + (3 + i) * kStageBox, l[i][0], l[i][1], l[i][2], l[i][3]);
        }
      } else if (EPI == PAIR_SWIGLU) {
        box_bf16(at, lane, 2 * h, v);
      } else {
        if (EPI != PAIR_SWIGLU_F32) scaled(v, box * kBox + h * 16);
        if (p.addend) {
#pragma unroll
          for (int j = 0; j < 2; j++) {
            uint4 a = make_uint4(0, 0, 0, 0);
            if (EPI == PAIR_BF16) a = ld_shared4(box_at(at, lane, 2 * h + j));
            else if (c0 + 8 * j < p.N) a = *reinterpret_cast<const uint4*>(p.addend + (size_t)row * p.N + c0 + 8 * j);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
              v[8 * j + 2 * i] = __float_as_uint(__uint_as_float(v[8 * j + 2 * i]) + bf16lo(w[i]));
              v[8 * j + 2 * i + 1] = __float_as_uint(__uint_as_float(v[8 * j + 2 * i + 1]) + bf16hi(w[i]));
            }
          }
        }
        if (kBox == 32) box_f32(at, lane, 4 * h, v);
        else box_bf16(at, lane, 2 * h, v);
      }
    }
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) {
      if (EPI == PAIR_SWIGLU) {
        tma_store_3d(&map_d, col0, row0, 0, at);
        if (p.keep) {
          tma_store_3d(&map_e, col0, row0, 0, at + kStageBox);
          tma_store_3d(&map_e, col0, row0, 1, at + 2 * kStageBox);
        }
      } else if (kGrad) {
        tma_store_3d(&map_e, col0, row0, 0, at);
        tma_store_3d(&map_e, col0, row0, 1, at + kStageBox);
        if (p.keep) tma_store_3d(&map_d, col0, row0, 0, at + 2 * kStageBox);
        if (kLo) {
          tma_store_3d(&map_e, col0, row0, 2, at + 3 * kStageBox);
          tma_store_3d(&map_e, col0, row0, 3, at + 4 * kStageBox);
          if (p.keep) tma_store_3d(&map_d, col0, row0, 1, at + 5 * kStageBox);
        }
      } else {
        const CUtensorMap* md = kTwo && tl.second ? &map_d2 : &map_d;
        if (EPI == PAIR_F32 && p.reduce) tma_add_3d(md, col0, row0, 0, at);
        else tma_store_3d(md, kBox == 32 ? 2 * col0 : col0, row0, 0, at);  // (an fp32 column is two of 2 bytes)
      }
      store_commit();
    }
  };

  const int per_q = p.ewarps >> 2;  // epilogue warps that share a quadrant of TMEM lanes, box by box
  if (warp >= 4 && ew < p.ewarps) {
    const int q = warp & 3, which = ew >> 2;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    Ring acc;
    for (int t = t_first; ok && t < ntiles; t += step, acc.next(2)) {
      const PairTile tl = pair_tile<kTwo>(p, t, cols);
      const int b = acc.slot;
      column_scales(tl);
      const float rs = row_scale(tl, q);
      const bool first = p.split == 1 && which < nbox && there(tl, which, q);
      if (asks && p.split > 1 && ew < 4 / p.split * nbox) {  // the first box that this warp joins
        const int mine = 4 / p.split, jq = part + p.split * (ew % mine), box = ew / mine;
        if (there(tl, box, jq)) ask(tl, box, jq);
      }
      if (asks && first) {
        ask(tl, which, q);
        if (kGrad && lane == 0)  // the others' on their way to L2
          for (int box = which + per_q; box < nbox && there(tl, box, q); box += per_q)
            for (int z = 0; z < 2; z++) tma_prefetch_3d(&map_g, tl.n0 + box * 64, tl.m0 + rank * 128 + q * 32, z);
      }
      if (!(ok = warp_wait(tfull(b), acc.parity, &s_abort))) break;
      tc_fence_after();
      const uint32_t d = tmem + b * 256 + lanes;
      if (p.split == 1) {
        for (int box = which; box < nbox && there(tl, box, q); box += per_q) {
          const bool more = asks && box + per_q < nbox && there(tl, box + per_q, q);
          if (kTurns && more) ask(tl, box + per_q, q);
          unit(tl, box, q, rs, [&](int c, uint32_t (&v)[16]) { tmem_ld16(d + c, v); }, [](uint32_t (&v)[16]) { tmem_wait16(v); });
          if (!kTurns && more) ask(tl, box + per_q, q);
        }
      } else {
        // the partial sums, [column][row], where the stages were: all are used
        for (int c = which * 16; c < p.bn; c += 16 * per_q) {
          uint32_t v[16];
          tmem_ld16(d + c, v);
          tmem_wait16(v);
          const uint32_t at = base + (uint32_t)(c * 128 + q * 32 + lane) * 4u;
#pragma unroll
          for (int j = 0; j < 16; j++)
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + j * 512), "r"(v[j]) : "memory");
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_rank(tempty(b), first_cta));
    }
  }
  if (p.split > 1) {
    // Part i joins the rows of the quadrants i, i + split, in the order of the parts, in its own
    // shared memory: no other reads them there. All threads come here, whatever became of
    // their waits; a cluster has one tile. (One 4-byte value at a time by the epilogue warps alone
    // took 10 us.)
    __syncwarp();
    cluster_sync();
    const int mine = 4 / p.split, all = p.bn * 8 * mine;  // 16 bytes each: 4 rows of a column
    auto place = [&](int i) {
      const int c = i / (8 * mine), r = i % (8 * mine), q = part + p.split * (r >> 3);
      return base + (uint32_t)(c * 128 + q * 32 + (r & 7) * 4) * 4u;
    };
    constexpr int kAtOnce = 3;  // (a load takes most of a microsecond)
    for (int i0 = tid; i0 < all; i0 += kAtOnce * kThreads) {
      float4 v[kAtOnce][kSplitMost];
#pragma unroll
      for (int k = 0; k < kAtOnce; k++) {
        const uint32_t at = place(min(i0 + k * kThreads, all - 1));
#pragma unroll
        for (int s = 0; s < kSplitMost; s++)
          if (s < p.split) v[k][s] = ld_cluster4(at, 2 * s + rank);
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; k++) {
        float4 sum = v[k][0];
#pragma unroll
        for (int s = 1; s < kSplitMost; s++)
          if (s < p.split) sum.x += v[k][s].x, sum.y += v[k][s].y, sum.z += v[k][s].z, sum.w += v[k][s].w;
        const int i = i0 + k * kThreads;
        if (i < all)
          st_shared4(place(i), __float_as_uint(sum.x), __float_as_uint(sum.y), __float_as_uint(sum.z), __float_as_uint(sum.w));
      }
    }
    __syncthreads();
    if (warp >= 4 && ew < p.ewarps) {
      const PairTile tl = pair_tile<kTwo>(p, min(t_first, ntiles - 1), cols);
      for (int i = ew; i < mine * nbox; i += p.ewarps) {
        const int q = part + p.split * (i % mine), box = i / mine;
        if (!there(tl, box, q)) continue;
        if (asks && i != ew) ask(tl, box, q);
        unit(tl, box, q, row_scale(tl, q), [&](int c, uint32_t (&v)[16]) { smem_ld16(base + (uint32_t)(c * 128 + q * 32 + lane) * 4u, v); }, [](uint32_t (&)[16]) {});
      }
    }
  }
  // (where a wait ended early, copies in flight land before the shared memory goes)
  for (; landed != asked; landed++)
    for (int i = 0; i < 1000 && !mbar_try_wait(loads(ew, landed & 1), (landed >> 1) & 1); i++) {
      }
  if (warp >= 4 && lane == 0) store_wait_all();  // shared memory is read and the results are written
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while the other's instructions or loads reach into it
  tc_fence_after();
  if (warp == 1) tmem_dealloc2(tmem, 512);
  // the status words: this CTA's, and from CTA 0 those that no CTA has, and the second launch's
  if (tid == 0 && (s_abort || !p.status_keep)) p.status[blockIdx.x] = s_abort;
  if (blockIdx.x == 0 && !p.status_keep)
    for (int i = gridDim.x + tid; i < 2 * kMaxSms; i += kThreads) p.status[i] = 0;
}

}  // namespace dense
}  // namespace moe
