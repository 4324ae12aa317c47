// Products of few rows of x (at most kStreamRows) with bf16 or int8 weights, for decoding.
//
// Every weight is used for a handful of rows: its bytes are the time. A warp holds 16 weight
// rows (the M side of mma.m16n8k16) and reads them straight into the operand registers, 16
// bytes a lane: the order of k within an instruction is free as long as both operands have
// the same one, so lane (g, i) takes the 16 bytes i of 64 from row g, without shared memory
// or shuffles. Rows of x are the N side, 8 at a time, from L1 and L2. With int8 weights and
// codes both operands are widened to fp16 in registers (exact: 1024 + 128 + v, less 1152), the
// products are exact in fp32. (IMMA runs at 274 multiplications a clock and SM on this GPU,
// fp16 at 1050: an SM's share of the HBM rate is 22 int8 weights a clock, times 8 rows each 176.)
//
// The warps of a CTA share its rows' K, chunk by chunk in turn, and join their sums through shared
// memory in warp order. With swiglu the 16 rows are 8 gate rows and the up rows of the same
// columns, so that one thread has both sums.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "dense_params.h"
#include "ptx.cuh"

namespace moe {
namespace dense {
namespace {

__device__ __forceinline__ uint4 ld_weights(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
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
__device__ __forceinline__ uint32_t sub_1152(uint32_t v) {
  const __half2 k = __half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&v), k);
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Four int8 -> four fp16: the byte v + 128 under the exponent of 1024 is 1152 + v.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  lo = sub_1152(__byte_perm(u, 0x64646464u, 0x4140));
  hi = sub_1152(__byte_perm(u, 0x64646464u, 0x4342));
}

constexpr int kMostWarps = 16;

// MT: 16-row blocks of weights a CTA, NT: 8-row blocks of x.
template <bool I8, int MT, int NT>
__global__ void __launch_bounds__(32 * kMostWarps) stream_kernel(const StreamParams p) {
  extern __shared__ float s_sums[];  // [warp][row of x][weight row]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
  const int g = lane >> 2, i = lane & 3;
  const int64_t row_bytes = (int64_t)p.K * (I8 ? 1 : 2);
  const int rows_out = (p.swiglu ? 8 : 16) * MT;  // results of a CTA for each row of x
  const int r0 = blockIdx.x * rows_out;

  const uint8_t* w[MT][2];
#pragma unroll
  for (int m = 0; m < MT; m++) {
    // (rows past the matrix repeat its last one; their sums are not used)
    const int lo = p.swiglu ? min(r0 + m * 8 + g, p.R - 1) : min(r0 + m * 16 + g, p.R - 1);
    const int hi = p.swiglu ? p.R + lo : min(r0 + m * 16 + g + 8, p.R - 1);
    w[m][0] = static_cast<const uint8_t*>(p.w) + lo * row_bytes + i * 16;
    w[m][1] = static_cast<const uint8_t*>(p.w) + hi * row_bytes + i * 16;
  }
  const uint8_t* x[NT];
#pragma unroll
  for (int n = 0; n < NT; n++)
    x[n] = static_cast<const uint8_t*>(p.x) + (int64_t)min(n * 8 + g, p.T - 1) * p.x_stride * (I8 ? 1 : 2) + i * 16;

  float acc[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; m++)
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
      for (int j = 0; j < 4; j++) acc[m][n][j] = 0.0f;

  const int64_t step = (int64_t)warps * 128;
  // the weights do not depend on the launch before: their first lines on their way
  for (int64_t at = warp * 128, c = 0; c < 4 && at < row_bytes; c++, at += step) {
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
      for (int h = 0; h < 2; h++)
        if ((i & 1) == 0 && at + i * 16 < row_bytes)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(w[m][h] + at + i * 16));
  }
  pdl_wait();
  pdl_launch_dependents();

  // A chunk is 128 bytes of every row, as two halves; what lies past a row is zero.
  constexpr int kUnroll = MT * NT <= 2 ? 2 : 1;
  for (int64_t at0 = warp * 128; at0 < row_bytes; at0 += kUnroll * step) {
    uint4 a[kUnroll][MT][2][2], b[kUnroll][NT][2];
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int v = 0; v < kUnroll; v++) {
      const int64_t at = at0 + v * step;
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const bool in = at + h * 64 + i * 16 < row_bytes;
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
          for (int r = 0; r < 2; r++) a[v][m][r][h] = in ? ld_weights(w[m][r] + at + h * 64) : zero;
#pragma unroll
        for (int n = 0; n < NT; n++)
          b[v][n][h] = in && n * 8 + g < p.T ? *reinterpret_cast<const uint4*>(x[n] + at + h * 64) : zero;
      }
    }
#pragma unroll
    for (int v = 0; v < kUnroll; v++)
#pragma unroll
      for (int h = 0; h < 2; h++) {
        if (I8) {
          auto word = [](const uint4& q, int j) { return j == 0 ? q.x : j == 1 ? q.y : j == 2 ? q.z : q.w; };
#pragma unroll
          for (int j = 0; j < 4; j++) {
            uint32_t al[MT][4];
#pragma unroll
            for (int m = 0; m < MT; m++) {
              widen4(word(a[v][m][0][h], j), al[m][0], al[m][2]);
              widen4(word(a[v][m][1][h], j), al[m][1], al[m][3]);
            }
#pragma unroll
            for (int n = 0; n < NT; n++) {
              uint32_t b0, b1;
              widen4(word(b[v][n][h], j), b0, b1);
#pragma unroll
              for (int m = 0; m < MT; m++) mma_f16(acc[m][n], al[m][0], al[m][1], al[m][2], al[m][3], b0, b1);
            }
          }
        } else {
#pragma unroll
          for (int n = 0; n < NT; n++)
#pragma unroll
            for (int m = 0; m < MT; m++) {
              const uint4 &lo = a[v][m][0][h], &hi = a[v][m][1][h], &xb = b[v][n][h];
              mma_bf16x(acc[m][n], lo.x, hi.x, lo.y, hi.y, xb.x, xb.y);
              mma_bf16x(acc[m][n], lo.z, hi.z, lo.w, hi.w, xb.z, xb.w);
            }
        }
      }
  }

  // [warp][column][weight row], columns 16 MT + 4 apart: no bank twice
  constexpr int kPitch = 16 * MT + 4;
  float* mine = s_sums + warp * (8 * NT * kPitch);
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
  for (int j = tid; j < rows_out * p.T; j += blockDim.x) {
    const int t = j / rows_out, r = j % rows_out, row = r0 + r;
    if (row >= p.R) continue;
    // swiglu: block r / 8's gate row r % 8, its up row 8 further on
    const float* at = s_sums + t * kPitch + (p.swiglu ? (r >> 3) * 16 + (r & 7) : r);
    float v = 0.0f, u = 0.0f;
    for (int k = 0; k < warps; k++) {
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
      v = v / (1.0f + expf(-v)) * u;
    }
    if (p.addend) v += __bfloat162float(p.addend[o]);
    if (p.out_f32) static_cast<float*>(p.out)[o] = v;
    else static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(v);
  }
  if (p.status && blockIdx.x == 0)  // this launch has no waits, and later ones only set words
    for (int j = tid; j < 2 * rows::kMaxSms; j += blockDim.x) p.status[j] = 0;
}

template <bool I8, int MT, int NT>
cudaError_t launch(const StreamParams& p, int warps, bool pdl, cudaStream_t s) {
  StreamParams q = p;
  cudaLaunchConfig_t c = {};
  const int rows_out = (p.swiglu ? 8 : 16) * MT;
  c.gridDim = dim3((unsigned)((p.R + rows_out - 1) / rows_out));
  c.blockDim = dim3(32 * warps);
  c.dynamicSmemBytes = (size_t)warps * 8 * NT * (16 * MT + 4) * 4;
  c.stream = s;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  c.attrs = a;
  c.numAttrs = 1;
  void* args[] = {&q};
  return cudaLaunchKernelExC(&c, reinterpret_cast<const void*>(&stream_kernel<I8, MT, NT>), args);
}

template <bool I8>
cudaError_t choose(const StreamParams& p, bool pdl, int sms, cudaStream_t s) {
  // fewer than two CTAs of 16 rows an SM: more warps share a CTA's K
  const int blocks = (p.R * (p.swiglu ? 2 : 1) + 15) / 16;
  const int warps = blocks < 2 * sms ? 16 : 8;
  if (p.T <= 8) return launch<I8, 1, 1>(p, warps, pdl, s);
  if (p.T <= 16) return launch<I8, 1, 2>(p, warps, pdl, s);
  // two blocks of weight rows read x half as often; not where that leaves SMs without a CTA
  if (blocks < 4 * sms) return launch<I8, 1, 4>(p, 8, pdl, s);
  return launch<I8, 2, 4>(p, 8, pdl, s);
}

}  // namespace

cudaError_t launch_stream(const StreamParams& p, bool int8, bool pdl, int sms, cudaStream_t s) {
  return int8 ? choose<true>(p, pdl, sms, s) : choose<false>(p, pdl, sms, s);
}

}  // namespace dense
}  // namespace moe
