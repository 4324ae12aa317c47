// Rows to 8-bit integers, and what the integer products need around them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/moe_decode_dense.h"
#include "dense_params.h"
#include "tc.cuh"

namespace moe {
namespace dense {
namespace {

// The code of v in a row of largest magnitude top (both scaled by the same power of two, so that
// 127 v neither overflows nor loses bits): 127 v / top to the nearest, halves to even.
// v * inv is off by a few steps of fp32, so at most the choice between two neighbours is open; what
// is left of 127 v after q tops decides. bf16: all terms have at most 16 bits and the
// difference is exact. fp32: it is exact in 64 bits, looked at only next to a half.
template <bool F32>
__device__ int code_of(float v, float top, float inv) {
  float q = rintf(v * inv);
  const float r = fmaf(-q, top, 127.0f * v), a = fabsf(r) * 2.0f;
  if (F32) {
    if (fabsf(a - top) <= top * 0x1p-14f) {
      const double d = 127.0 * v - (double)q * top, m = fabs(d) * 2.0;
      if (m > top || (m == top && (static_cast<int>(q) & 1))) q += d > 0.0 ? 1.0f : -1.0f;
    }
  } else if (a > top || (a == top && (static_cast<int>(q) & 1))) {
    q += r > 0.0f ? 1.0f : -1.0f;
  }
  return static_cast<int>(q);
}

// In most rows neither scaling nor that is asked for: v inv + 1.5 2^23 in one rounding has the nearest whole
// number in its low bits, and v inv's distance from it says whether a half is near. (The whole of code_of
// for every value: 128 us for 134 million fp32 values, where the bytes take 99.)
constexpr float kWhole = 12582912.0f, kNearHalf = 0.4999f;

// A chunk is 8 elements: 16 bytes of bf16 or 32 of fp32.
template <bool F32>
struct Chunk;
template <>
struct Chunk<false> {
  uint4 d;
  __device__ void load(const void* row, int c) { d = static_cast<const uint4*>(row)[c]; }
  __device__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
    for (int j = 0; j < 4; j++) v[2 * j] = bf16lo(w[j]), v[2 * j + 1] = bf16hi(w[j]);
  }
};
template <>
struct Chunk<true> {
  float4 a, b;
  __device__ void load(const void* row, int c) {
    a = static_cast<const float4*>(row)[2 * c];
    b = static_cast<const float4*>(row)[2 * c + 1];
  }
  __device__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};

constexpr int64_t kManyRows = 512;
constexpr int kKept = 4;  // chunks of a thread that stay in registers between the two passes

// G threads a row, of 256 a CTA: about four chunks each.
template <bool F32, bool HALF, int G>
__global__ void __launch_bounds__(256) quantise_kernel(const uint8_t* x, int64_t stride_bytes, int64_t rows, int inner,
                                                       void* codes, float* scale) {
  __shared__ float s_top[8];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, me = tid % G;
  const int64_t row = (int64_t)blockIdx.x * (256 / G) + tid / G;
  const bool mine = row < rows;
  const uint8_t* src = x + row * stride_bytes;
  const int chunks = mine ? inner / 8 : 0;
  Chunk<F32> kept[kKept];
  float top = 0.0f;
  bool odd = false;  // a NaN (maximum passes over it)
  auto look = [&](const Chunk<F32>& c) {
    float v[8];
    c.get(v);
#pragma unroll
    for (int j = 0; j < 8; j++) {
      top = fmaxf(top, fabsf(v[j]));
      odd |= v[j] != v[j];
    }
  };
#pragma unroll
  for (int k = 0; k < kKept; k++)
    if (me + k * G < chunks) kept[k].load(src, me + k * G);
#pragma unroll
  for (int k = 0; k < kKept; k++)
    if (me + k * G < chunks) look(kept[k]);
  for (int c = me + kKept * G; c < chunks; c += G) {
    Chunk<F32> v;
    v.load(src, c);
    look(v);
  }
  if (odd) top = INFINITY;
  // magnitudes are ordered as their bits are
  uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
  if (G > 32) {
    if (lane == 0) s_top[tid >> 5] = __uint_as_float(bits);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < G / 32; k++) bits = max(bits, __float_as_uint(s_top[(tid & ~(G - 1)) / 32 + k]));
  }
  top = __uint_as_float(bits);
  const bool bad = !(top < INFINITY), none = top == 0.0f;
  if (me == 0 && mine) scale[row] = bad ? __uint_as_float(0x7fffffffu) : __fdiv_rn(top, 127.0f);
  // a power of two that keeps 127 v and 127 / top inside fp32
  const float pre = top > 0x1p100f ? 0x1p-32f : top < 0x1p-60f ? 0x1p64f : 1.0f;
  const float pre2 = top < 0x1p-100f ? 0x1p30f : 1.0f;  // (top may be as small as 2^-149)
  const float t = bad || none ? 1.0f : top * pre * pre2;
  const float inv = 127.0f / t;
  const bool plain = pre == 1.0f && pre2 == 1.0f && !bad && !none;
  auto store = [&](const Chunk<F32>& c, int at) {
    float v[8];
    c.get(v);
    float q[8];
    bool near = !plain;
    if (plain) {
#pragma unroll
      for (int j = 0; j < 8; j++) {
        q[j] = fmaf(v[j], inv, kWhole) - kWhole;
        near |= fabsf(fmaf(v[j], inv, -q[j])) > kNearHalf;
      }
    }
    if (near && plain && !F32) {
      // halves are common among bf16 numbers: the exact remainder decides, as in code_of
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const float r = fmaf(-q[j], t, 127.0f * v[j]), a = fabsf(r) * 2.0f;
        if (a > t || (a == t && (__float_as_uint(q[j] + kWhole) & 1))) q[j] += copysignf(1.0f, r);
      }
    } else if (near) {
#pragma unroll
      for (int j = 0; j < 8; j++) q[j] = bad || none ? 0.0f : (float)code_of<F32>(v[j] * pre * pre2, t, inv);
    }
    if (HALF) {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const __half2 h = __floats2half2_rn(q[2 * j], q[2 * j + 1]);
        o[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
      reinterpret_cast<uint4*>(static_cast<__half*>(codes) + row * inner)[at] = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
      auto four = [&](int j) {  // the low bytes of q + 1.5 2^23
        const uint32_t w[4] = {__float_as_uint(q[j] + kWhole), __float_as_uint(q[j + 1] + kWhole), __float_as_uint(q[j + 2] + kWhole),
                               __float_as_uint(q[j + 3] + kWhole)};
        return __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
      };
      reinterpret_cast<uint2*>(static_cast<int8_t*>(codes) + row * inner)[at] = make_uint2(four(0), four(4));
    }
  };
#pragma unroll
  for (int k = 0; k < kKept; k++)
    if (me + k * G < chunks) store(kept[k], me + k * G);
  for (int c = me + kKept * G; c < chunks; c += G) {
    Chunk<F32> v;
    v.load(src, c);
    store(v, c);
  }
}

// 16 codes a thread.
__global__ void __launch_bounds__(256) widen_kernel(const int8_t* src, int64_t stride, int64_t count, int cols, __half* dst) {
  pdl_wait();
  pdl_launch_dependents();
  const int per = cols / 16;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count * per; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / per;
    const int c = (int)(i - r * per);
    const uint4 v = *reinterpret_cast<const uint4*>(src + r * stride + c * 16);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 4; j++) rows::int8x4_f16x4(w[j], o[2 * j], o[2 * j + 1]);
    uint4* to = reinterpret_cast<uint4*>(dst + r * cols + c * 16);
    to[0] = make_uint4(o[0], o[1], o[2], o[3]);
    to[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

__global__ void __launch_bounds__(256) zero_kernel(uint4* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = make_uint4(0, 0, 0, 0);
}

cudaError_t launch_with(const void* f, int64_t blocks, void** args, bool pdl, cudaStream_t s) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)blocks);
  c.blockDim = dim3(256);
  c.stream = s;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  c.attrs = a;
  c.numAttrs = 1;
  return cudaLaunchKernelExC(&c, f, args);
}

template <bool F32, bool HALF>
const void* quantise_fn(int g) {
  return g == 32   ? reinterpret_cast<const void*>(&quantise_kernel<F32, HALF, 32>)
         : g == 64 ? reinterpret_cast<const void*>(&quantise_kernel<F32, HALF, 64>)
         : g == 128 ? reinterpret_cast<const void*>(&quantise_kernel<F32, HALF, 128>)
                    : reinterpret_cast<const void*>(&quantise_kernel<F32, HALF, 256>);
}

}  // namespace

cudaError_t launch_quantise(int dtype, const void* x, int64_t x_stride, int64_t rows, int inner, void* codes, bool half,
                            float* scale, bool pdl, cudaStream_t s) {
  const bool f32 = dtype == MOE_F32;
  const uint8_t* src = static_cast<const uint8_t*>(x);
  int64_t bytes = x_stride * (f32 ? 4 : 2);
  // Many rows: as many threads as keep a row between them. (16384 rows of 2048 bf16 values with 256 threads a row,
  // one chunk each: 43 us.) Few: a row's latency counts, and all 256 share it.
  int g = 256;
  if (rows >= kManyRows)
    while (g > 32 && inner <= 8 * (g / 2) * kKept) g /= 2;
  const void* f = f32 ? (half ? quantise_fn<true, true>(g) : quantise_fn<true, false>(g))
                      : (half ? quantise_fn<false, true>(g) : quantise_fn<false, false>(g));
  void* args[] = {&src, &bytes, &rows, &inner, &codes, &scale};
  return launch_with(f, (rows + 256 / g - 1) / (256 / g), args, pdl, s);
}

cudaError_t launch_widen(const int8_t* src, int64_t stride, int64_t rows, int cols, __half* dst, bool pdl, cudaStream_t s) {
  const int64_t n = rows * (cols / 16), blocks = (n + 255) / 256;
  void* args[] = {&src, &stride, &rows, &cols, &dst};
  return launch_with(reinterpret_cast<const void*>(&widen_kernel), blocks < 152 * 16 ? blocks : 152 * 16, args, pdl, s);
}

cudaError_t launch_zero(void* p, int64_t bytes, cudaStream_t s) {
  uint4* q = static_cast<uint4*>(p);
  int64_t n = bytes / 16;
  void* args[] = {&q, &n};
  const int64_t blocks = (n + 255) / 256;
  return launch_with(reinterpret_cast<const void*>(&zero_kernel), blocks < 152 * 8 ? blocks : 152 * 8, args, false, s);
}

}  // namespace dense
}  // namespace moe
