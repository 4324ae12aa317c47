// What the host code of the many-row and of the dense operators shares: checks of
// addresses and overlaps, the device, tensor-map encoding, errors. (static, not inline: an
// inline function's static variables are one for all libraries of a process.)
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "../../include/moe_decode.h"
#include "rows_params.h"

namespace moe {
namespace rows {

constexpr int64_t kMaxRows = (int64_t)1 << 24;  // rows of one call
constexpr int kStatusKernels = 2;               // sets of status words at a workspace's start

static inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
static inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
// Whether the bytes at a share any with those at b.
static inline bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const intptr_t d = static_cast<const char*>(b) - static_cast<const char*>(a);
  return a && b && d < a_bytes && -d < b_bytes;
}
// Whether rows of `width` bytes every `stride` bytes share any with those at out.
static inline bool rows_overlap(const void* x, int64_t stride, int64_t width, int64_t rows, const void* out, int64_t bytes) {
  const intptr_t d = static_cast<const char*>(out) - static_cast<const char*>(x);
  if (d + bytes <= 0) return false;
  const int64_t last = std::min(rows - 1, (d + bytes - 1) / stride);  // the last row that starts before out's end
  return last * stride + width > d;
}
static inline size_t up(size_t v, size_t a) { return (v + a - 1) / a * a; }
static inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static inline EncodeTiled encode_tiled() {
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

struct Device {
  int sms = 0, smem = 0, id = 0;
};
static inline bool device(Device* d) {
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

static inline moe_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  cudaGetLastError();  // the error is reported here, not by a later call
  return MOE_ERR_CUDA;
}

}  // namespace rows
}  // namespace moe
