// Products of few rows of x (at most kStreamRows) with bf16 or int8 weights, for decoding.
//
// Every weight is used for a handful of rows: its bytes are the time. A warp holds 16 weight
// rows (the M side of mma.m16n8k16), rows of x are the N side, 8 at a time. The order of k within
// an instruction is free as long as both operands have the same one, so lane (g, i) takes the 16
// bytes i of 64 of row g: it copies them to shared memory with cp.async and reads the same
// bytes back, so that a ring of copies needs no barrier and no registers (loads into registers, the
// same operands: 22.6 us for 67 MB of int8 weights where this takes 16.5, 15.9 for 67 MB of
// bf16 where this takes 14.4; prefetches to L2 before them were slower). With int8 weights and
// codes both operands are widened to fp16 in registers, exactly; the products are exact in fp32.
// (IMMA runs at 274 multiplications a clock and SM on this GPU, fp16 at 1050: an SM's share of the
// HBM rate is 22 int8 weights a clock, times 8 rows 176.)
//
// The warps of a CTA share its rows' K, chunk by chunk in turn, and join their sums through shared
// memory in warp order; copies of the next block of rows are under way meanwhile. With swiglu
// the 16 rows are 8 gate rows and the up rows of the same columns, so that one thread has both sums.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "dense_params.h"
#include "tc.cuh"

namespace moe {
namespace dense {
namespace {

// 16 bytes of global memory to shared memory, or zeros; weights pass by L1, rows of x stay in it.
__device__ __forceinline__ void copy_weights(uint32_t dst, const uint8_t* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_rows(uint32_t dst, const uint8_t* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 ld_shared4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16x(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kWarps = 8;
constexpr int pieces(int mt, int nt, int halves, bool lo) { return (2 * mt + (lo ? 2 : 1) * nt) * halves; }
constexpr int sums_floats(int mt, int nt) { return kWarps * 8 * nt * (16 * mt + 4); }
constexpr int stream_smem(int mt, int nt, int halves, int stages, bool lo) {
  return kWarps * stages * pieces(mt, nt, halves, lo) * 512 + 2 * sums_floats(mt, nt) * 4;
}

// MT: 16-row blocks of weights, NT: 8-row blocks of x, HALVES: 64-byte pieces of a row in a stage, LO: x is
// the sum of two bf16 numbers.
template <bool I8, int MT, int NT, int HALVES, int STAGES, bool LO>
__global__ void __launch_bounds__(32 * kWarps) stream_kernel(const StreamParams p) {
  extern __shared__ __align__(16) uint8_t s_raw[];
  constexpr int kPieces = pieces(MT, NT, HALVES, LO), kPitch = 16 * MT + 4, kChunk = 64 * HALVES;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, i = lane & 3;
  const int64_t row_bytes = (int64_t)p.K * (I8 ? 1 : 2);
  const int rows_out = (p.swiglu ? 8 : 16) * MT;  // results of a block for each row of x
  const int blocks = (p.R + rows_out - 1) / rows_out;
  const int chunks = (int)((row_bytes + kChunk - 1) / kChunk);
  const uint32_t ring = smem_u32(s_raw) + warp * (STAGES * kPieces * 512) + lane * 16;
  float* sums = reinterpret_cast<float*>(s_raw + kWarps * STAGES * kPieces * 512);

  // What this warp copies next: chunk ic of block ib, into stage is.
  int ib = blockIdx.x, ic = warp, is = 0;
  auto copy = [&](int b, int c, int s, bool weights, bool rows) {
    const int64_t at = (int64_t)c * kChunk + i * 16;
    const uint32_t dst = ring + s * (kPieces * 512);
#pragma unroll
    for (int h = 0; h < HALVES; h++) {
      const bool in = at + h * 64 < row_bytes;
      if (weights) {
#pragma unroll
        for (int m = 0; m < MT; m++) {
          // (rows past the matrix repeat its last one; their sums are not used)
          const int lo = min(b * rows_out + (p.swiglu ? m * 8 : m * 16) + g, p.R - 1);
          const int hi = p.swiglu ? p.R + lo : min(b * rows_out + m * 16 + g + 8, p.R - 1);
          const uint8_t* w = static_cast<const uint8_t*>(p.w) + at + h * 64;
          copy_weights(dst + ((h * MT + m) * 2) * 512, in ? w + lo * row_bytes : static_cast<const uint8_t*>(p.w), in);
          copy_weights(dst + ((h * MT + m) * 2 + 1) * 512, in ? w + hi * row_bytes : static_cast<const uint8_t*>(p.w), in);
        }
      }
      if (rows) {
#pragma unroll
        for (int n = 0; n < NT; n++) {
          const bool there = in && n * 8 + g < p.T;
          copy_rows(dst + (2 * MT * HALVES + h * NT + n) * 512,
                    static_cast<const uint8_t*>(p.x) + (there ? (int64_t)(n * 8 + g) * p.x_stride * (I8 ? 1 : 2) + at + h * 64 : 0), there);
          if (LO)
            copy_rows(dst + ((2 * MT + NT) * HALVES + h * NT + n) * 512,
                      reinterpret_cast<const uint8_t*>(p.x_lo) + (there ? (int64_t)(n * 8 + g) * p.x_stride * 2 + at + h * 64 : 0), there);
        }
      }
    }
  };
  auto next = [&]() {
    is = is + 1 == STAGES ? 0 : is + 1;
    ic += kWarps;
    if (ic >= chunks) {
      ic = warp;
      ib += gridDim.x;
    }
  };
  const bool any = warp < chunks;  // (a warp without chunks has zeros to add)
  // the weights do not depend on the launch before
  {
    int b = ib, c = ic;
#pragma unroll
    for (int s = 0; s < STAGES - 1; s++) {
      if (any && b < blocks) copy(b, c, s, true, false);
      c += kWarps;
      if (c >= chunks) c = warp, b += gridDim.x;
    }
  }
  pdl_wait();
  pdl_launch_dependents();
#pragma unroll
  for (int s = 0; s < STAGES - 1; s++) {
    if (any && ib < blocks) copy(ib, ic, s, false, true);
    copies_commit();
    next();
  }

  int stage = 0, buf = 0;
  for (int b = blockIdx.x; b < blocks; b += gridDim.x, buf ^= 1) {
    float acc[MT][NT][4];
    float rest[MT][NT][4];  // LO: the products of the second numbers
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
      for (int n = 0; n < NT; n++)
#pragma unroll
        for (int j = 0; j < 4; j++) acc[m][n][j] = rest[m][n][j] = 0.0f;
    for (int c = warp; c < chunks; c += kWarps) {
      copies_wait<STAGES - 2>();
      const uint32_t src = ring + stage * (kPieces * 512);
      stage = stage + 1 == STAGES ? 0 : stage + 1;
#pragma unroll
      for (int h = 0; h < HALVES; h++) {
        // (a lane reads back what it copied itself)
        uint4 a[MT][2], x[NT];
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
          for (int r = 0; r < 2; r++) a[m][r] = ld_shared4(src + ((h * MT + m) * 2 + r) * 512);
#pragma unroll
        for (int n = 0; n < NT; n++) x[n] = ld_shared4(src + (2 * MT * HALVES + h * NT + n) * 512);
        if (I8) {
          auto word = [](const uint4& q, int j) { return j == 0 ? q.x : j == 1 ? q.y : j == 2 ? q.z : q.w; };
#pragma unroll
          for (int j = 0; j < 4; j++) {
            uint32_t al[MT][4];
#pragma unroll
            for (int m = 0; m < MT; m++) {
              rows::int8x4_f16x4(word(a[m][0], j), al[m][0], al[m][2]);
              rows::int8x4_f16x4(word(a[m][1], j), al[m][1], al[m][3]);
            }
#pragma unroll
            for (int n = 0; n < NT; n++) {
              uint32_t b0, b1;
              rows::int8x4_f16x4(word(x[n], j), b0, b1);
#pragma unroll
              for (int m = 0; m < MT; m++) mma_f16(acc[m][n], al[m][0], al[m][1], al[m][2], al[m][3], b0, b1);
            }
          }
        } else {
#pragma unroll
          for (int n = 0; n < NT; n++)
#pragma unroll
            for (int m = 0; m < MT; m++) {
              mma_bf16x(acc[m][n], a[m][0].x, a[m][1].x, a[m][0].y, a[m][1].y, x[n].x, x[n].y);
              mma_bf16x(acc[m][n], a[m][0].z, a[m][1].z, a[m][0].w, a[m][1].w, x[n].z, x[n].w);
            }
          if (LO) {
#pragma unroll
            for (int n = 0; n < NT; n++) {
              const uint4 l = ld_shared4(src + ((2 * MT + NT) * HALVES + h * NT + n) * 512);
#pragma unroll
              for (int m = 0; m < MT; m++) {
                mma_bf16x(rest[m][n], a[m][0].x, a[m][1].x, a[m][0].y, a[m][1].y, l.x, l.y);
                mma_bf16x(rest[m][n], a[m][0].z, a[m][1].z, a[m][0].w, a[m][1].w, l.z, l.w);
              }
            }
          }
        }
      }
      if (ib < blocks) copy(ib, ic, is, true, true);
      copies_commit();
      next();
    }

    // (where the first numbers' products are infinite, the second ones', of any sign, would make NaN of them)
    if (LO) {
#pragma unroll
      for (int m = 0; m < MT; m++)
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
          for (int j = 0; j < 4; j++)
            if (fabsf(acc[m][n][j]) < INFINITY) acc[m][n][j] += rest[m][n][j];
    }
    // [warp][row of x][weight row], rows of x 16 MT + 4 apart: no bank twice. Two buffers in turn: one
    // barrier a block.
    float* mine = sums + buf * sums_floats(MT, NT) + warp * (8 * NT * kPitch);
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
      for (int n = 0; n < NT; n++) {
        float* at = mine + (n * 8 + 2 * i) * kPitch + m * 16 + g;
        at[0] = acc[m][n][0];
        at[kPitch] = acc[m][n][1];
        at[8] = acc[m][n][2];
        at[kPitch + 8] = acc[m][n][3];
      }
    __syncthreads();
    for (int j = tid; j < rows_out * p.T; j += 32 * kWarps) {
      const int t = j / rows_out, r = j % rows_out, row = b * rows_out + r;
      if (row >= p.R) continue;
      // swiglu: block r / 8's gate row r % 8, its up row 8 further on
      const float* at = sums + buf * sums_floats(MT, NT) + t * kPitch + (p.swiglu ? (r >> 3) * 16 + (r & 7) : r);
      float v = 0.0f, u = 0.0f;
#pragma unroll
      for (int k = 0; k < kWarps; k++) {
        v += at[k * (8 * NT * kPitch)];
        if (p.swiglu) u += at[k * (8 * NT * kPitch) + 8];
      }
      if (I8) {
        const float s = p.x_scale[t];
        v *= s * __ldg(p.w_scale + row);
        if (p.swiglu) u *= s * __ldg(p.w_scale + p.R + row);
      }
      const int64_t o = (int64_t)t * p.R + row;
      if (p.swiglu) {
        if (p.keep) {
          p.keep[o + (int64_t)t * p.R] = __float2bfloat16_rn(v);
          p.keep[o + (int64_t)(t + 1) * p.R] = __float2bfloat16_rn(u);
        }
        v = rows::silu_mul_f32(v, u);
      }
      if (p.addend) v += __bfloat162float(p.addend[o]);
      if (p.out_f32) static_cast<float*>(p.out)[o] = v;
      else if (p.out_lo) {
        const __nv_bfloat16 hi = __float2bfloat16_rn(rows::high(v));
        static_cast<__nv_bfloat16*>(p.out)[o] = hi;
        p.out_lo[o] = __float2bfloat16_rn(rows::low(v, __bfloat162float(hi)));
      } else {
        static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(v);
      }
    }
  }
  copies_wait<0>();
  if (p.status && blockIdx.x == 0)  // this launch has no waits, and later ones only set words
    for (int j = tid; j < 2 * rows::kMaxSms; j += 32 * kWarps) p.status[j] = 0;
}

// PER_SM: CTAs of an SM. All are resident at once: one that started behind another would find its ring empty.
template <bool I8, int MT, int NT, int HALVES, int STAGES, int PER_SM, bool LO = false>
cudaError_t launch(const StreamParams& p, bool pdl, int sms, cudaStream_t s) {
  const void* f = reinterpret_cast<const void*>(&stream_kernel<I8, MT, NT, HALVES, STAGES, LO>);
  constexpr int smem = stream_smem(MT, NT, HALVES, STAGES, LO);
  static_assert(PER_SM * (smem + 1024) <= 228 * 1024, "the SM's shared memory, 1 KB of it for the system in each CTA");
  static std::atomic<uint64_t> ready{0};  // devices whose limit is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev);
  }
  StreamParams q = p;
  cudaLaunchConfig_t c = {};
  const int rows_out = (p.swiglu ? 8 : 16) * MT, blocks = (p.R + rows_out - 1) / rows_out;
  c.gridDim = dim3((unsigned)(blocks < sms * PER_SM ? blocks : sms * PER_SM));
  c.blockDim = dim3(32 * kWarps);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  c.attrs = a;
  c.numAttrs = 1;
  void* args[] = {&q};
  return cudaLaunchKernelExC(&c, f, args);
}

// Stages and CTAs an SM: up to 8 rows the fastest for matrices of 17 to 134 MB, of 1 to 4 CTAs and 2 to 6 stages of 64 or
// 128 bytes a row. More rows of x take two blocks of weight rows a CTA, which read them half as often; the ring
// and the sums of one such CTA fill an SM. (16 rows, int8, 4096 to 2 x 4800: 12.6 us; with CTAs that waited for one another's
// end 13.9; two CTAs of three stages 11.3, but 13.0 for 11.4 from 8192 to 4096.)
template <bool I8>
cudaError_t choose(const StreamParams& p, bool pdl, int sms, cudaStream_t s) {
  if (p.T <= 8) return launch<I8, 1, 1, 2, 4, 2>(p, pdl, sms, s);
  return launch<I8, 2, 2, 1, 4, 1>(p, pdl, sms, s);
}

}  // namespace

cudaError_t launch_stream(const StreamParams& p, bool int8, bool pdl, int sms, cudaStream_t s) {
  if (p.x_lo) {  // (bf16, at most kExactRows)
    return p.T <= 8 ? launch<false, 1, 1, 1, 5, 2, true>(p, pdl, sms, s) : launch<false, 2, 2, 1, 4, 1, true>(p, pdl, sms, s);
  }
  return int8 ? choose<true>(p, pdl, sms, s) : choose<false>(p, pdl, sms, s);
}

}  // namespace dense
}  // namespace moe
