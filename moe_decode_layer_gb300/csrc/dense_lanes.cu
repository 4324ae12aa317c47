// Some rows times bf16 or int8 weights (tcgen05, sm_103a): D [R, T] = W X^T, bf16 or fp16 operands, fp32
// accumulators, and out = D^T, with scales, as the block has them.
//
// The weights take the tensor core's lanes and the rows of x its columns, so that a step costs what
// the rows are (the pair product's tile of 256 rows costs the same for 32). A CTA has 128 rows of
// weights (gate and up: 64 and 64) and all of x. Codes: TMA brings 128 of each weight row and the
// same k of x as fp16; a thread widens a weight row, exactly, and puts it into tensor memory, from where the
// tensor core takes it: what shared memory moves for a weight are its byte in and its byte out.
// Few tiles: the CTAs of a cluster take parts of K, and their sums are joined through distributed
// shared memory, in the order of the parts.
//
// What bounds it: the weights' bytes; int8 0.30 us for a step of 128 k in 128 CTAs (7 TB/s), behind 8 us of start and end
// with the rows' codes: 32 rows, 4096 to 2 x 8192 (67 MB), 20.1 us (with both operands widened in
// registers for mma.sync 32, as a pair product 30), 8192 to 4096 14.3 (17 and 29), 128 rows 27.1 and 19.5 (pairs 31.5 and 30.3).
// bf16: the 4096 x 8192 block of 16 rows in 37.8 us (201 MB, 5.3 TB/s), of 128 in 47.0 (52.6 as a pair product).
// (Joined by loads from the other CTAs and another barrier, instead of stores to them: 1 to 2 us more.)
//
// Warps: 0 copies, 1 tensor core, 2 tensor memory, 4..11 widen (four take a step, four the next one)
// and read the sums; all write results. The weights' first copies are under way before the launch that
// makes x has ended: it does not write weights, and all before it have ended. Every wait is
// bounded; who gives up sets a flag that the others look at, and the CTA's status word.
#include <algorithm>
#include <atomic>

#include "dense_gemm.cuh"

namespace moe {
namespace dense {
namespace {

constexpr int kThreads = 384, kSlots = 12, kStages = 6;
constexpr int kWeightBytes = 16384;  // of a slot: 128 rows of 128 bytes

template <bool I8>
__global__ void __launch_bounds__(kThreads, 1)
    lanes_kernel(const __grid_constant__ LaneParams p, const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ __align__(8) uint64_t s_bar[3 * kSlots + 2 * kStages + 2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bar0 = smem_u32(s_bar);
  uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
  const float4* sums = reinterpret_cast<const float4*>(smem + p.sums_off);
  float* s_weights = reinterpret_cast<float*>(smem + p.scale_off);  // scales: [128], [T]
  float* s_rows = s_weights + 128;
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kSlots + s); };
  auto ready = [&](int a) { return bar0 + 8u * (2 * kSlots + a); };
  auto used = [&](int a) { return bar0 + 8u * (2 * kSlots + kStages + a); };
  auto rows = [&](int s) { return bar0 + 8u * (2 * kSlots + 2 * kStages + s); };
  const uint32_t done = bar0 + 8u * (3 * kSlots + 2 * kStages), drain = done + 8u;
  const int part = cluster_rank(), tile = blockIdx.x / p.split;
  constexpr int kStep = I8 ? 128 : 64, kBoxes = I8 ? 2 : 1;  // k of a step; boxes of rows of x
  const int ksteps = (p.K + kStep - 1) / kStep, k0 = ksteps * part / p.split, n = ksteps * (part + 1) / p.split - k0;
  const int x_box = p.cols * 128;
  const uint32_t slot_bytes = kWeightBytes + kBoxes * x_box;

  if (tid == 0) {
    s_abort = 0;
    for (int s = 0; s < kSlots; s++) mbar_init(full(s), 1), mbar_init(rows(s), 1), mbar_init(empty(s), 1);
    for (int a = 0; a < kStages; a++) mbar_init(ready(a), 4), mbar_init(used(a), 1);
    mbar_init(done, 1);
    mbar_init(drain, 1);
    mbar_init_fence();
    tma_prefetch_map(&map_w);
    tma_prefetch_map(&map_x);
  }
  auto weights = [&](int i, int s) {
    mbar_arrive_expect_tx(full(s), kWeightBytes);
    const int k = (k0 + i) * kStep;
    for (int h = 0; h < 2; h++)
      tma_load_3d(base + s * slot_bytes + h * 8192, &map_w, k, p.swiglu ? tile * 64 : tile * 128 + h * 64, p.swiglu ? h : 0, full(s));
  };
  const int first = min(p.slots, n);
  if (tid == 0)
    for (int i = 0; i < first; i++) weights(i, i);
  if (warp == 2) {
    tmem_alloc(smem_u32(&s_tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  // (its wait: before others' memory is written)
  const bool early = p.sums_off != 0;
  if (p.split > 1 && (early || warp < 4)) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  // (widening does not wait for the codes of x)
  auto behind = [&] {
    pdl_wait();
    fence_proxy_async_global();
    pdl_launch_dependents();
  };
  if (!I8 || warp < 4) behind();

  bool ok = true;
  if (warp == 0) {
    // ---------------------------------------------------------------- copies
    if (lane == 0) {
      Ring it;
      for (int i = 0; i < n; i++, it.next(p.slots)) {
        const uint32_t s = it.slot;
        if (i >= first) {
          if (!(ok = wait_phase(empty(s), it.parity ^ 1, &s_abort))) break;
          weights(i, s);
        }
        mbar_arrive_expect_tx(rows(s), kBoxes * x_box);
        for (int h = 0; h < kBoxes; h++)
          tma_load_3d(base + s * slot_bytes + kWeightBytes + h * x_box, &map_x, (k0 + i) * kStep + h * 64, 0, 0, rows(s));
      }
      ok = ok && wait_phase(done, 0, &s_abort);  // then all have landed
      if (!ok) {  // let the copies in flight land before the shared memory goes
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < kDrainNs) __nanosleep(1000);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- tensor core
    const bool leader = elect_one();
    Ring it, at;
    for (int i = 0; i < n; i++, it.next(p.slots), at.next(p.stages)) {
      if (!(ok = warp_wait(I8 ? ready(at.slot) : full(it.slot), I8 ? at.parity : it.parity, &s_abort) && warp_wait(rows(it.slot), it.parity, &s_abort))) break;
      tc_fence_after();
      const uint32_t w = base + it.slot * slot_bytes, x = w + kWeightBytes;
      if (leader) {
#pragma unroll
        for (int j = 0; j < kStep / 16; j++) {
          const uint64_t rows_of_x = smem_desc(x + (j >> 2) * x_box) + 2 * (j & 3);
          if (I8) mma_bf16_ta(tmem, tmem + p.stage_at + at.slot * 64 + 8 * j, rows_of_x, p.idesc, i != 0 || j != 0);
          else mma_bf16(tmem, smem_desc(w) + 2 * j, rows_of_x, p.idesc, i != 0 || j != 0);
        }
        mma_commit(empty(it.slot));
        if (I8) mma_commit(used(at.slot));
      }
      __syncwarp();
    }
    if (leader) {
      mma_commit(ok ? done : drain);
      if (!ok) {
        const uint64_t t0 = global_ns();
        while (!mbar_try_wait(drain, 0) && global_ns() - t0 < kDrainNs) {
        }
      }
    }
    __syncwarp();
  } else if (warp < 4) {
    // ---------------------------------------------------------------- scales, and addends on their way
    const int me = tid - 64;
    for (int j = me; I8 && j < 128; j += 64) {
      const int h = p.swiglu && j >= 64, r = p.swiglu ? tile * 64 + (j & 63) : tile * 128 + j;
      s_weights[j] = r < p.R ? __ldg(p.w_scale + h * p.R + r) : 0.0f;
    }
    for (int j = me; I8 && j < p.T; j += 64) s_rows[j] = p.x_scale[j];
    if (p.addend)
      for (int t = part + p.split * me; t < p.T; t += p.split * 64)
        for (int r = tile * 128; r < min(tile * 128 + 128, p.R); r += 64)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(p.addend + (int64_t)t * p.R + r));
  } else {
    // ---------------------------------------------------------------- widening, then the sums
    const int row = (warp & 3) * 32 + lane, group = (warp - 4) >> 2;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    Ring it, at;
    auto wait = [&](LaneWait what, uint32_t s, uint32_t parity) { return warp_wait(what == LANE_FULL ? full(s) : empty(s), parity, &s_abort); };
    for (int i = 0; I8 && i < n; i++, it.next(p.slots), at.next(p.stages)) {
      if ((i & 1) != group) continue;
      if (!(ok = landed(it, p.slots, p.stages, wait))) break;
      const uint32_t src = base + it.slot * slot_bytes + row * 128;
      uint32_t o[2][32];
#pragma unroll
      for (int h = 0; h < 2; h++)
#pragma unroll
        for (int c = 0; c < 4; c++) {
          const uint4 q = ld_shared4(src + (((h * 4 + c) ^ (row & 7)) << 4));
          const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int j = 0; j < 4; j++) int8x4_f16x4(w[j], o[h][8 * c + 2 * j], o[h][8 * c + 2 * j + 1]);
        }
      if (i == behind_at(p.stages, group)) behind();
      if (!(ok = warp_wait(used(at.slot), at.parity ^ 1, &s_abort))) break;
      tc_fence_after();
      const uint32_t to = tmem + lanes + p.stage_at + at.slot * 64;
      tmem_st32(to, o[0]);
      tmem_st32(to + 32, o[1]);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ready(at.slot), 1);
    }
    if (I8 && n <= behind_at(p.stages, group)) behind();
    if (p.split > 1 && early) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    ok = ok && warp_wait(done, 0, &s_abort);  // all slots are used
    if (p.split > 1 && !early) {
      asm volatile("barrier.cluster.arrive.release;" ::: "memory");
      asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    }
    // Row t of x is part t % split's: it gets [t / split][part][weight row] from every part.
    if (ok) {
      tc_fence_after();
      for (int c = group * 8; c < p.cols; c += 16) {
        uint32_t v[8];
        tmem_ld8(tmem + lanes + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 8; j++) {
          const int to = (c + j) & (p.split - 1);
          const uint32_t at = map_rank(base + p.sums_off + (c + j - to + part) * 512 + row * 4, to);
          if (c + j < p.T) asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v[j]) : "memory");
        }
      }
      tc_fence_before();
    }
  }
  if (p.split > 1 && warp < 4) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  __syncwarp();
  if (p.split > 1) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(tmem, 512);

  // Part i writes the rows of x i, i + split, ...: four results a thread.
  const int groups = p.swiglu ? 16 : 32, mine = (p.T - part + p.split - 1) / p.split;
  for (int i = tid; i < mine * groups; i += kThreads) {
    const int t = part + p.split * (i / groups), g = i % groups, o = tile * groups * 4 + g * 4;
    if (o >= p.R) continue;
    const float4* at = sums + (t - part) * 32 + g;
    float v[4] = {}, u[4] = {};
    for (int s = 0; s < p.split; s++) {
      const float4 a = at[s * 32];
      v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
      if (p.swiglu) {
        const float4 b = at[s * 32 + 16];
        u[0] += b.x, u[1] += b.y, u[2] += b.z, u[3] += b.w;
      }
    }
    const int64_t to = (int64_t)t * p.R + o;
    if (!I8 && p.keep) {
      __nv_bfloat16* keep = p.keep + to + (int64_t)t * p.R;
      *reinterpret_cast<uint2*>(keep) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
      *reinterpret_cast<uint2*>(keep + p.R) = make_uint2(pack_bf16(u[0], u[1]), pack_bf16(u[2], u[3]));
    }
    const float xs = I8 ? s_rows[t] : 1.0f;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      if (I8) v[j] *= xs * s_weights[g * 4 + j];
      if (I8) u[j] *= xs * s_weights[(64 + g * 4 + j) & 127];
      if (p.swiglu) v[j] = silu_mul_f32(v[j], u[j]);
    }
    if (p.addend) {
      const uint2 a = *reinterpret_cast<const uint2*>(p.addend + to);
      v[0] += bf16lo(a.x), v[1] += bf16hi(a.x), v[2] += bf16lo(a.y), v[3] += bf16hi(a.y);
    }
    if (p.out_f32) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + to) = make_float4(v[0], v[1], v[2], v[3]);
    else *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + to) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  }
  if (tid == 0 && (s_abort || !p.status_keep)) p.status[blockIdx.x] = s_abort;
  if (blockIdx.x == 0 && !p.status_keep)
    for (int i = gridDim.x + tid; i < 2 * kMaxSms; i += kThreads) p.status[i] = 0;
}

}  // namespace

// CTAs of a cluster: as many as fill the SMs, where clusters of that size fit (of 152 SMs 76, 36 and 15).
int lanes_split(int tiles, int ksteps, int sms) {
  return tiles <= sms / 10 && ksteps >= 16 ? 8 : tiles <= sms * 9 / 38 && ksteps >= 8 ? 4 : tiles <= sms / 2 && ksteps >= 4 ? 2 : 1;
}

cudaError_t launch_lanes(LaneParams p, bool int8, const CUtensorMap& w, const CUtensorMap& x, int dev, int smem, int sms, cudaStream_t s) {
  const void* k = int8 ? reinterpret_cast<const void*>(&lanes_kernel<true>) : reinterpret_cast<const void*>(&lanes_kernel<false>);
  static std::atomic<uint64_t> known[2];  // devices whose limit is set
  std::atomic<uint64_t>& ready = known[int8];
  if (dev >= 64 || !(ready.load() >> dev & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem - 1024);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev);
  }
  const int tiles = lanes_tiles(p.R, p.swiglu);
  p.split = lanes_split(tiles, (p.K + (int8 ? 127 : 63)) / (int8 ? 128 : 64), sms);
  p.scale_off = smem - 4 * 1024;
  // (Sums of few rows have a place of their own: they are handed over a microsecond earlier, without a
  // wait for the other CTAs' slots. Of many, that would cost a slot or two.)
  p.sums_off = p.split > 1 && p.cols <= 64 ? p.scale_off - p.cols * 512 : 0;
  p.slots = std::min(kSlots, (p.sums_off ? p.sums_off : p.scale_off) / (kWeightBytes + (int8 ? 2 : 1) * p.cols * 128));
  p.stage_at = (p.cols + 63) / 64 * 64;
  p.stages = std::min(kStages, (512 - p.stage_at) / 64);
  // fp32 accumulators, fp16 or bf16 operands, M = 128
  p.idesc = 1u << 4 | (int8 ? 0u : 1u << 7 | 1u << 10) | (uint32_t)(p.cols >> 3) << 17 | 8u << 24;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)(tiles * p.split));
  c.blockDim = dim3(kThreads);
  // All of the SM's shared memory: a CTA takes all tensor memory, and may not wait for what a CTA of another launch
  // holds while those of its cluster wait for it.
  c.dynamicSmemBytes = smem - 1024;
  c.stream = s;
  cudaLaunchAttribute a[2];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = p.pdl;
  a[1].id = cudaLaunchAttributeClusterDimension;
  a[1].val.clusterDim.x = p.split;
  a[1].val.clusterDim.y = a[1].val.clusterDim.z = 1;
  c.attrs = a;
  c.numAttrs = 2;
  CUtensorMap mw = w, mx = x;
  void* args[] = {&p, &mw, &mx};
  return cudaLaunchKernelExC(&c, k, args);
}

}  // namespace dense
}  // namespace moe
