"""The library's host code over a stand-in for the CUDA runtime (CPU only).

The objects that the library is linked from are linked again with a runtime that
keeps a list of the launches, checks tensor maps by the documented rules and can
fail at a chosen call. Nothing runs on a device: device addresses are plain numbers.
"""

import ctypes
import os
import subprocess

from moe_decode_layer_gb300 import _lib, build

STUB = r"""
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>
#include <cstring>
#include <string>
#include <unordered_map>
#include <vector>

namespace {
struct Launch { std::string name; unsigned grid, cluster; size_t smem; int pdl; };
std::vector<Launch> g_launches;
std::unordered_map<const void*, std::string> g_names;
std::unordered_map<const void*, int> g_smem;
cudaError_t g_last = cudaSuccess;
int g_fail_encode = -1, g_fail_launch = -1, g_encodes = 0, g_tries = 0, g_bad_maps = 0;
int g_capturing = 0;
size_t g_read = 0;
struct Config { dim3 grid, block; size_t smem; cudaStream_t stream; } g_config;

cudaError_t launch(const void* f, dim3 grid, size_t smem, unsigned cluster, int pdl) {
  if (g_tries++ == g_fail_launch || smem > 48 * 1024 && smem > (size_t)g_smem[f] || grid.x % cluster)
    return g_last = cudaErrorLaunchOutOfResources;
  g_launches.push_back({g_names[f], grid.x, cluster, smem, pdl});
  return cudaSuccess;
}

CUresult encode(CUtensorMap*, CUtensorMapDataType t, cuuint32_t rank, void* base, const cuuint64_t* dims,
                const cuuint64_t* strides, const cuuint32_t* box, const cuuint32_t*, CUtensorMapInterleave,
                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  if (g_encodes++ == g_fail_encode) return CUDA_ERROR_INVALID_VALUE;
  const unsigned size = t == CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 ? 2 : 1;
  bool ok = (uintptr_t)base % 16 == 0 && box[0] * size == 128;
  for (unsigned i = 0; i < rank; i++) ok = ok && dims[i] > 0 && dims[i] <= 1ull << 32 && box[i] >= 1 && box[i] <= 256;
  for (unsigned i = 0; i + 1 < rank; i++) ok = ok && strides[i] % 16 == 0 && strides[i] < 1ull << 40;
  g_bad_maps += !ok;
  return ok ? CUDA_SUCCESS : CUDA_ERROR_INVALID_VALUE;
}
}  // namespace

extern "C" {
void** __cudaRegisterFatBinary(void*) { static void* h; return &h; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* host, char*, const char* name, int, uint3*, uint3*, dim3*, dim3*, int*) {
  g_names[host] = name;
}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
unsigned __cudaPushCallConfiguration(dim3 g, dim3 b, size_t s, cudaStream_t st) { g_config = {g, b, s, st}; return 0; }
cudaError_t __cudaPopCallConfiguration(dim3* g, dim3* b, size_t* s, void* st) {
  *g = g_config.grid, *b = g_config.block, *s = g_config.smem;
  *(cudaStream_t*)st = g_config.stream;
  return cudaSuccess;
}
cudaError_t __cudaGetKernel(cudaKernel_t* k, const void* f) { *k = (cudaKernel_t)f; return cudaSuccess; }
cudaError_t __cudaLaunchKernel(cudaKernel_t k, dim3 g, dim3, void**, size_t s, cudaStream_t) { return launch((const void*)k, g, s, 1, 0); }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  unsigned cluster = 1;
  int pdl = 0;
  for (unsigned i = 0; i < c->numAttrs; i++) {
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) cluster = c->attrs[i].val.clusterDim.x;
    if (c->attrs[i].id == cudaLaunchAttributeProgrammaticStreamSerialization)
      pdl = c->attrs[i].val.programmaticStreamSerializationAllowed;
  }
  return launch(f, c->gridDim, c->dynamicSmemBytes, cluster, pdl);
}
cudaError_t cudaGetLastError() { const cudaError_t e = g_last; g_last = cudaSuccess; return e; }
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrMultiProcessorCount ? 152 : 227 * 1024;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute, int v) { g_smem[f] = v; return cudaSuccess; }
cudaError_t cudaMemcpyAsync(void* d, const void*, size_t n, cudaMemcpyKind, cudaStream_t) { g_read = n; memset(d, 0, n); return cudaSuccess; }
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus* s) { *s = (cudaStreamCaptureStatus)g_capturing; return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** f, unsigned, unsigned long long, cudaDriverEntryPointQueryResult* r) {
  *f = (void*)encode;
  *r = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}

void fake_reset(int fail_encode, int fail_launch, int pending) {
  g_launches.clear();
  g_fail_encode = fail_encode, g_fail_launch = fail_launch, g_last = (cudaError_t)pending;
  g_encodes = g_tries = g_bad_maps = 0;
}
void fake_capture(int on) { g_capturing = on, g_read = 0; }
int fake_launches() { return (int)g_launches.size(); }
const char* fake_name(int i) { return g_launches[i].name.c_str(); }
unsigned fake_grid(int i) { return g_launches[i].grid; }
int fake_pdl(int i) { return g_launches[i].pdl; }
int fake_encodes() { return g_encodes; }
int fake_bytes_read() { return (int)g_read; }
int fake_bad_maps() { return g_bad_maps; }
int fake_pending() { return (int)g_last; }
}
"""


def make(folder) -> ctypes.CDLL:
    """The library's many-row entry points over the stand-in, built in ``folder``."""
    build.build()
    objs = [os.path.join(build.BUILD, s.replace(".cu", ".o")) for s in build.ROWS_SOURCES]
    if not all(os.path.exists(o) for o in objs):  # a library that was brought along without its objects
        build.build(force=True)
    src, out = os.path.join(folder, "stub.cpp"), os.path.join(folder, "librows_fake.so")
    with open(src, "w") as f:
        f.write(STUB)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-O1", "-w", "-Wl,-Bsymbolic", "-I", cuda, src, *objs, "-o", out],
                   check=True)
    lib = ctypes.CDLL(out)
    real = _lib.load()
    for name in _lib.EXPORTS:
        if hasattr(lib, name):
            getattr(lib, name).argtypes, getattr(lib, name).restype = getattr(real, name).argtypes, ctypes.c_int32
    lib.fake_name.restype = ctypes.c_char_p
    return lib
