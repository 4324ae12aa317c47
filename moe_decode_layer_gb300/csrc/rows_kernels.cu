// The small kernels around the grouped product: bringing the rows of each group
// together, and the weighted sum over a row's experts.
#include <cooperative_groups.h>

#include "rows_kernels.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace moe {
namespace rows {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanCtas = 8;  // CTAs (one cluster) for long lists

// Inclusive scan over the block's 1024 threads; warp_sums holds 32 ints.
__device__ __forceinline__ int block_scan(int v, int* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += o;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  return v + (warp ? warp_sums[warp - 1] : 0);
}

// Counting sort in one launch: the CTAs of a cluster each count a part of the
// pairs, read one another's counts through distributed shared memory, and give
// out positions from their own part of each group. The order inside a group is that
// of the atomics; no result depends on it (a row's sums are its own, and the
// combine finds them through pos). 8008 pairs of 512 experts: 7 us; bound by its
// chain of passes and barriers.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p) {
  __shared__ int s_count[kMaxGroups + 1];
  __shared__ int s_next[kMaxGroups + 1];
  __shared__ int s_warp[32];
  cg::cluster_group cl = cg::this_cluster();
  pdl_launch_dependents();
  const int tid = threadIdx.x, nc = cl.num_blocks(), me = cl.block_rank();
  const int G = p.groups + (p.keep_none ? 1 : 0);  // the last one: none
  for (int g = tid; g <= p.groups; g += kPlanThreads) s_count[g] = 0;
  __syncthreads();
  const int per = (p.pairs + nc - 1) / nc;
  const int b = min(p.pairs, me * per), e = min(p.pairs, b + per);
  for (int i = b + tid; i < e; i += kPlanThreads) {
    const int g = __ldg(p.idx + i);
    const bool ok = (unsigned)g < (unsigned)p.groups;
    if (ok || p.keep_none) atomicAdd(&s_count[ok ? g : p.groups], 1);
  }
  if (nc > 1) cl.sync(); else __syncthreads();
  // one thread per group (at most 1024 and "none")
  int total = 0, mine = 0;
  if (tid < G) {
    for (int c = 0; c < nc; c++) {
      const int v = nc > 1 ? cl.map_shared_rank(s_count, c)[tid] : s_count[tid];
      if (c < me) mine += v;
      total += v;
    }
  }
  const int room = tid < p.groups ? (total + p.align - 1) & -p.align : total;
  const int end = block_scan(room, s_warp);
  const int start = end - room;
  if (me == 0 && tid < p.groups)
    for (int i = total; i < room; i++) p.src_row[start + i] = -1;
  if (tid < G) s_next[tid] = start + mine;
  // "none" of 1024 adapters is thread 1024's: every pair that is left
  if (p.keep_none && G > kPlanThreads && tid == kPlanThreads - 1) {
    int m = 0;
    for (int c = 0; c < me; c++) m += cl.map_shared_rank(s_count, c)[kPlanThreads];  // me = 0: none
    s_next[kPlanThreads] = end + m;
  }
  __syncthreads();
  for (int i = b + tid; i < e; i += kPlanThreads) {
    const int g = __ldg(p.idx + i);
    const bool ok = (unsigned)g < (unsigned)p.groups;
    int at = -1;
    if (ok || p.keep_none) {
      at = atomicAdd(&s_next[ok ? g : p.groups], 1);
      p.src_row[at] = i / p.per_row;
    }
    if (p.pos) p.pos[i] = at;
  }
  if (me == 0) {
    if (tid < p.groups) {
      p.off[tid] = start;
      if (tid == p.groups - 1) p.off[p.groups] = end;
    }
    if (p.keep_none) {
      if (tid == p.groups) p.off[p.groups + 1] = end;
      if (p.groups == kPlanThreads && tid == kPlanThreads - 1) {
        int none = 0;
        for (int c = 0; c < nc; c++) none += nc > 1 ? cl.map_shared_rank(s_count, c)[kPlanThreads] : s_count[kPlanThreads];
        p.off[p.groups + 1] = end + none;
      }
    }
    if (p.ents) {
      // the shared groups' tiles first: they are the longest
      const int sb = (p.rows + p.nmax - 1) / p.nmax;
      for (int i = tid; i < p.shared * sb; i += kPlanThreads) {
        const int s = i / sb, t = i % sb;
        p.ents[i] = pack_tile(p.groups + s, p.pairs + s * p.rows + t * p.nmax, min(p.nmax, p.rows - t * p.nmax), t, sb);
      }
      const int n = tid < p.groups ? total : 0;
      const int nb = (n + p.nmax - 1) / p.nmax;
      const int last = block_scan(nb, s_warp);
      const int first = p.shared * sb + last - nb;
      for (int t = 0; t < nb; t++)
        p.ents[first + t] = pack_tile(tid, start + t * p.nmax, min(p.nmax, n - t * p.nmax), t, nb);
      if (tid == kPlanThreads - 1) *p.nent = p.shared * sb + last;
    }
  }
  if (nc > 1) cl.sync();  // no CTA leaves while another reads its counts
}

constexpr int kSpreadWarps = 8;

// One warp per position; the grouped product then copies its rows in boxes. Bound by
// the bytes written (and read from L2): 65536 positions of 2048 columns, 0.30 GB, 54 us.
__global__ void __launch_bounds__(kSpreadWarps * 32)
    spread_kernel(const __nv_bfloat16* __restrict__ x, int64_t x_stride, const int* src_row, const int* count,
                  int inner, __nv_bfloat16* __restrict__ dst) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t at = (int64_t)blockIdx.x * kSpreadWarps + (threadIdx.x >> 5);
  if (at >= *count) return;
  const int row = src_row[at];
  if (row < 0) return;
  const uint4* s = reinterpret_cast<const uint4*>(x + (int64_t)row * x_stride);
  uint4* d = reinterpret_cast<uint4*>(dst + at * inner);
  const int n = inner / 8;
  int i = threadIdx.x & 31;
  for (; i + 96 < n; i += 128) {
    const uint4 a = __ldg(s + i), b = __ldg(s + i + 32), c = __ldg(s + i + 64), e = __ldg(s + i + 96);
    d[i] = a;
    d[i + 32] = b;
    d[i + 64] = c;
    d[i + 96] = e;
  }
  for (; i < n; i += 32) d[i] = __ldg(s + i);
}

constexpr int kShrinkWarps = 8;

// One warp per (row, rank column): the adapter's row and the row of x, 16 bytes a
// lane and load. For few rows: bound by the latency of one pass over K (32 rows, rank
// 16, K = 2560: 7 us from cold caches).
__global__ void __launch_bounds__(kShrinkWarps * 32)
    shrink_kernel(const __nv_bfloat16* __restrict__ x, int64_t x_stride, const __nv_bfloat16* __restrict__ a,
                  const float* __restrict__ scale, const int* __restrict__ ids, float* __restrict__ u, int inner,
                  int rank, int adapters) {
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, j = blockIdx.y * kShrinkWarps + (threadIdx.x >> 5);
  const int64_t t = blockIdx.x;
  const int id = __ldg(ids + t);
  if (j >= rank || (unsigned)id >= (unsigned)adapters) return;
  const uint4* ap = reinterpret_cast<const uint4*>(a + ((size_t)id * rank + j) * inner);
  const uint4* xp = reinterpret_cast<const uint4*>(x + t * x_stride);
  float acc[2] = {0.0f, 0.0f};
  const int n = inner / 8;
  int i = lane;
#pragma unroll 4
  for (; i + 32 < n; i += 64) {
    const uint4 a0 = __ldg(ap + i), a1 = __ldg(ap + i + 32), x0 = __ldg(xp + i), x1 = __ldg(xp + i + 32);
    dot8_bf16(acc[0], a0, x0);
    dot8_bf16(acc[1], a1, x1);
  }
  if (i < n) dot8_bf16(acc[0], __ldg(ap + i), __ldg(xp + i));
  float v = acc[0] + acc[1];
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if (lane == 0) u[t * rank + j] = scale ? __ldg(scale + id) * v : v;
}

constexpr int kCombineThreads = 256;

// One thread per 4 columns of a row; y is fp32 and every y row is read once. Bound by
// those bytes: 8192 rows of 9 x 2048, 0.67 GB in all, 109 us (6.1 TB/s). In bf16 they
// would halve, and add the rounding of each of a row's terms to the sum's.
__global__ void __launch_bounds__(kCombineThreads)
    combine_kernel(const float* y, const int* pos, const float* __restrict__ w,
                   const void* residual, bool residual_f32, __nv_bfloat16* out, int rows, int hidden, int top_k, int shared) {
  pdl_wait();
  const int cols = hidden / 4;
  const int64_t i = (int64_t)blockIdx.x * kCombineThreads + threadIdx.x;
  if (i >= (int64_t)rows * cols) return;
  const int t = (int)(i / cols), c = (int)(i % cols) * 4;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (residual && residual_f32) {
    a = *reinterpret_cast<const float4*>(static_cast<const float*>(residual) + (size_t)t * hidden + c);
  } else if (residual) {
    const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(residual) + (size_t)t * hidden + c);
    a = make_float4(bf16lo(r.x), bf16hi(r.x), bf16lo(r.y), bf16hi(r.y));
  }
#pragma unroll 4
  for (int j = 0; j < top_k; j++) {
    const int at = pos[(size_t)t * top_k + j];  // (pos and y are of the launches before: plain loads)
    const float f = __ldg(w + (size_t)t * top_k + j);
    if (at >= 0) {
      const float4 v = *reinterpret_cast<const float4*>(y + (size_t)at * hidden + c);
      a.x = fmaf(f, v.x, a.x);
      a.y = fmaf(f, v.y, a.y);
      a.z = fmaf(f, v.z, a.z);
      a.w = fmaf(f, v.w, a.w);
    }
  }
  for (int s = 0; s < shared; s++) {
    const float4 v =
        *reinterpret_cast<const float4*>(y + ((size_t)rows * top_k + (size_t)s * rows + t) * hidden + c);
    a.x += v.x;
    a.y += v.y;
    a.z += v.z;
    a.w += v.w;
  }
  uint2 o;
  o.x = f32_to_bf16_bits(a.x) | ((uint32_t)f32_to_bf16_bits(a.y) << 16);
  o.y = f32_to_bf16_bits(a.z) | ((uint32_t)f32_to_bf16_bits(a.w) << 16);
  *reinterpret_cast<uint2*>(out + (size_t)t * hidden + c) = o;
}

}  // namespace

cudaError_t launch_plan(const PlanParams& p, cudaStream_t s) {
  cudaLaunchConfig_t c = {};
  const int ctas = p.pairs > 2048 ? kPlanCtas : 1;
  c.gridDim = dim3(ctas);
  c.blockDim = dim3(kPlanThreads);
  c.stream = s;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeClusterDimension;
  a[0].val.clusterDim.x = ctas;
  a[0].val.clusterDim.y = a[0].val.clusterDim.z = 1;
  c.attrs = a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, plan_kernel, p);
}

cudaError_t launch_spread(const __nv_bfloat16* x, int64_t x_stride, const int* src_row, const int* count,
                          int64_t positions, int inner, __nv_bfloat16* dst, cudaStream_t s) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)((positions + kSpreadWarps - 1) / kSpreadWarps));
  c.blockDim = dim3(kSpreadWarps * 32);
  c.stream = s;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, spread_kernel, x, x_stride, src_row, count, inner, dst);
}

cudaError_t launch_shrink(const __nv_bfloat16* x, int64_t x_stride, const __nv_bfloat16* a, const float* scale,
                          const int* ids, float* u, int rows, int inner, int rank, int adapters, cudaStream_t s) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)rows, (unsigned)((rank + kShrinkWarps - 1) / kShrinkWarps));
  c.blockDim = dim3(kShrinkWarps * 32);
  c.stream = s;
  return cudaLaunchKernelEx(&c, shrink_kernel, x, x_stride, a, scale, ids, u, inner, rank, adapters);
}

cudaError_t launch_combine(const float* y, const int* pos, const float* w, const void* residual, bool residual_f32,
                           __nv_bfloat16* out, int rows, int hidden, int top_k, int shared, cudaStream_t s) {
  cudaLaunchConfig_t c = {};
  const int64_t n = (int64_t)rows * (hidden / 4);
  c.gridDim = dim3((unsigned)((n + kCombineThreads - 1) / kCombineThreads));
  c.blockDim = dim3(kCombineThreads);
  c.stream = s;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, combine_kernel, y, pos, w, residual, residual_f32, out, rows, hidden, top_k, shared);
}

}  // namespace rows
}  // namespace moe
