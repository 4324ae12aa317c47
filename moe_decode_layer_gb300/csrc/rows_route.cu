// Routing of any number of rows: one warp per row, the row's logits in registers.
//
// The choice is made on 32-bit keys and costs few instructions:
//   1. each lane's largest key; K rounds of a warp maximum over the 32 lane maxima
//      (each round retires the lanes that hold it) give a lower bound on the K-th
//      largest key;
//   2. the keys at or above the bound (about K of them) are listed in shared
//      memory; each is ranked against the others, one lane per candidate.
// Without a bias the order is the logits' own and exact. Where the keys are rounded
// values (a bias, sums over groups), neighbours in the order that are closer than
// their rounding errors, and not equal inputs, are decided in fp64: sums over groups
// without a bias by the groups' two logits, one lane each; sigmoid keys by the
// candidates' keys alone or the two groups at the border; else the row's whole choice by
// the definition. That is rare, and makes the choice independent of how the scores were
// computed. (fp64 runs
// at 1/64 of the fp32 rate: one row decided as a whole takes longer than all the
// others of a 4096-row launch, so the bounds below count each rounding.)
//
// One row takes 4 us, a launch's latency. 65536 rows of 512 logits (138 MB) take
// 39 us: 570 instructions a row, most on the integer pipe, where the bytes need 20.
// 4096 rows of 256 with a bias and groups take 12 us: 1460 instructions a row (a quotient
// and an exp for every expert, a shared-memory round for the groups' best keys, loops over
// the groups) on 27 rows an SM, which fill 55 to 60 % of the issue slots.
#include <cuda_bf16.h>

#include <cfloat>
#include <cmath>

#include "ptx.cuh"
#include "rows_kernels.h"

namespace moe {
namespace rows {
namespace {

constexpr int kWarps = 4;     // rows per CTA
constexpr int kCand = 64;     // candidates listed per row
constexpr int kMostK = 16;
constexpr float kMasked = -0x1.2ced34p+126f;  // the first fp32 at or below -1e38
constexpr float kLeast = -0x1.2ced32p+126f;   // the next one above it
constexpr float kLargest = 3e38f;

struct RouteParams {
  const void* logits;
  int64_t stride;
  const float* bias;
  int64_t rows;
  int32_t* idx;
  float* w;
  int E, K;
  int softmax;     // else sigmoid
  int groups, kept, best, group_size;
  uint32_t group_magic;  // 2^32 / group_size, rounded up
  int renormalise;
  float scale;
};

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(v);
  else return v;
}

// NaN and masks -> -inf; +inf and the like -> a finite value, so that no sum is NaN.
__device__ __forceinline__ float clean(float l) { return l > kMasked ? fminf(l, kLargest) : -INFINITY; }

__device__ __forceinline__ int group_of(const RouteParams& p, int e) {
  return p.group_size == 1 ? e : (int)__umulhi((uint32_t)e, p.group_magic);  // e < 1024: exact
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {  // not for NaN
  return order_key_f32(warp_max_u32(f32_order_key(v)));
}

__device__ __forceinline__ double sigmoid64(double l) { return 1.0 / (1.0 + exp(-l)); }

// The row's choice by the definition, in fp64 (there is a bias). src: the row's logits;
// key: E doubles of shared memory. Lane j < K returns its expert or -1.
template <typename T>
__device__ __noinline__ int choose64(const RouteParams& p, const T* src, double* key, int lane) {
  const int E = p.E;
  auto l = [&](int e) { return clean(to_f32(src[e])); };
  double norm = 1.0, top = 0.0;
  if (p.softmax) {
    float m = -INFINITY;
    for (int e = lane; e < E; e += 32) m = fmaxf(m, l(e));
    top = (double)warp_max(m);
    double s = 0.0;
    for (int e = lane; e < E; e += 32)
      if (l(e) > kMasked) s += exp((double)l(e) - top);
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    norm = s;
  }
  for (int e = lane; e < E; e += 32) {
    double v = -INFINITY;
    if (l(e) > kMasked) {
      v = p.softmax ? exp((double)l(e) - top) / norm : sigmoid64((double)l(e));
      v += (double)__ldg(p.bias + e);
    }
    key[e] = v;
  }
  __syncwarp();
  uint32_t keep = 0xffffffffu;
  if (p.kept < p.groups) {
    double v = -INFINITY;
    if (lane < p.groups) {
      double b1 = -INFINITY, b2 = -INFINITY;
      for (int i = 0; i < p.group_size; i++) {
        const double x = key[lane * p.group_size + i];
        if (x > b1) {
          b2 = b1;
          b1 = x;
        } else if (x > b2) {
          b2 = x;
        }
      }
      v = b1;
      if (p.best == 2 && b2 > -INFINITY) v += b2;
    }
    int rank = 0;
    for (int g = 0; g < p.groups; g++) {
      const double o = __shfl_sync(0xffffffffu, v, g);
      rank += o > v || (o == v && g < lane);
    }
    keep = __ballot_sync(0xffffffffu, lane < p.groups && rank < p.kept);
  }
  int mine = -1;
  for (int j = 0; j < p.K; j++) {
    double b = -INFINITY;
    int at = E;
    for (int e = lane; e < E; e += 32) {
      const double x = key[e];
      if (x > b && (keep >> group_of(p, e) & 1)) {
        b = x;
        at = e;
      }
    }
    for (int d = 16; d; d >>= 1) {
      const double ob = __shfl_xor_sync(0xffffffffu, b, d);
      const int oa = __shfl_xor_sync(0xffffffffu, at, d);
      if (ob > b || (ob == b && oa < at)) {
        b = ob;
        at = oa;
      }
    }
    if (lane == j && at < E) mine = at;
    __syncwarp();
    if (at < E && lane == 0) key[at] = -INFINITY;
    __syncwarp();
  }
  return mine;
}

// Where this lane's group (b1, b2: its two largest logits, or -inf; sub lanes a group) comes
// among the sums of two scores, in fp64. Without a bias; softmax scores times the row's
// common factor.
__device__ __noinline__ int group_rank64(const RouteParams& p, float b1, float b2, float top, int g, int sub) {
  auto score = [&](float l) { return p.softmax ? exp((double)l - (double)top) : sigmoid64((double)l); };  // -inf: 0
  const double v = b1 > -INFINITY ? score(b1) + score(b2) : -INFINITY;
  int rank = 0;
  for (int o = 0; o < p.groups; o++) {
    const double x = __shfl_sync(0xffffffffu, v, o * sub);
    rank += x > v || (x == v && o < g);
  }
  return rank;
}

// Whether group b's value comes before group a's, in fp64: half a warp each. Sigmoid
// scores with a bias.
template <typename T>
__device__ __noinline__ bool border64(const RouteParams& p, const T* src, int a, int b, int lane) {
  const int g = lane < 16 ? a : b;
  double b1 = -INFINITY, b2 = -INFINITY;
  for (int i = lane & 15; i < p.group_size; i += 16) {
    const int e = g * p.group_size + i;
    const float l = clean(to_f32(src[e]));
    const double x = l > kMasked ? fmax(sigmoid64((double)l) + (double)__ldg(p.bias + e), -INFINITY) : -INFINITY;
    b2 = fmax(b2, fmin(b1, x));
    b1 = fmax(b1, x);
  }
  for (int d = 8; d; d >>= 1) {
    const double o1 = __shfl_xor_sync(0xffffffffu, b1, d), o2 = __shfl_xor_sync(0xffffffffu, b2, d);
    b2 = fmax(fmax(b2, o2), fmin(b1, o1));
    b1 = fmax(b1, o1);
  }
  const double v = p.best == 2 && b2 > -INFINITY ? b1 + b2 : b1;
  const double va = __shfl_sync(0xffffffffu, v, 0), vb = __shfl_sync(0xffffffffu, v, 16);
  return vb > va || (vb == va && b < a);
}

// The row's choice by K warp maxima over the logits: when so many tie at the bound
// that they cannot all be listed. keep: bits of the groups in the choice.
template <typename T>
__device__ __noinline__ int choose_rounds(const RouteParams& p, const T* src, uint32_t keep, int lane) {
  int mine = -1;
  uint32_t last = 0xffffffffu;  // the key and expert chosen last: later ones come after it
  int last_e = -1;
  for (int r = 0; r < p.K; r++) {
    uint32_t b = 0;
    int at = 0x7fffffff;
    for (int e = lane; e < p.E; e += 32) {
      const float l = clean(to_f32(src[e]));
      if (!(l > kMasked) || !(keep >> group_of(p, e) & 1u)) continue;
      const uint32_t k = f32_order_key(l + 0.0f);
      if ((k < last || (k == last && e > last_e)) && k > b) {
        b = k;
        at = e;
      }
    }
    const uint32_t m = warp_max_u32(b);
    if (m == 0) break;
    last = m;
    last_e = __reduce_min_sync(0xffffffffu, b == m ? at : 0x7fffffff);
    if (lane == r) mine = last_e;
  }
  return mine;
}

struct Cand {
  uint32_t key;
  int e;
  float l;
};

// Whether fp32 keys cannot tell x from y, which comes after it: their rounding errors
// together reach their difference, and their inputs are not equal.
__device__ __forceinline__ bool confusable(const RouteParams& p, const Cand& x, const Cand& y, float tol_s) {
  const float a = order_key_f32(x.key), b = order_key_f32(y.key);
  const bool same = x.l == y.l && __ldg(p.bias + x.e) == __ldg(p.bias + y.e);
  return !same && a - b <= tol_s + 0x1p-22f * fmaxf(fabsf(a), fabsf(b));
}

// N: logits per lane (32 N >= E). VEC: 4 consecutive logits per lane and load.
// KEYS: there is a bias, or groups (else the choice is by the logits alone, whose
// order is the scores').
template <typename T, int N, bool VEC, bool KEYS>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ __align__(16) uint8_t s_dyn[];  // KEYS: per warp E doubles
  __shared__ uint64_t s_order[kWarps][kCand];  // key, then the complement of the expert: larger comes first
  __shared__ float s_logit[kWarps][kCand];
  __shared__ Cand s_sorted[kWarps][kMostK];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = (int64_t)blockIdx.x * kWarps + warp;
  if (row >= p.rows) return;
  const int E = p.E, K = p.K;
  auto at = [&](int j) { return VEC ? (j >> 2) * 128 + lane * 4 + (j & 3) : j * 32 + lane; };

  float l[N];
  const T* src = reinterpret_cast<const T*>(p.logits) + row * p.stride;
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      const int e = at(j);
      if (e < E) {  // E % 4 == 0
        if constexpr (sizeof(T) == 4) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(src + e));
          l[j] = v.x;
          l[j + 1] = v.y;
          l[j + 2] = v.z;
          l[j + 3] = v.w;
        } else {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(src + e));
          l[j] = bf16lo(v.x);
          l[j + 1] = bf16hi(v.x);
          l[j + 2] = bf16lo(v.y);
          l[j + 3] = bf16hi(v.y);
        }
      } else {
        l[j] = l[j + 1] = l[j + 2] = l[j + 3] = -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; j++) l[j] = at(j) < E ? to_f32(src[at(j)]) : -INFINITY;
  }
  const bool bias = KEYS && p.bias;
  const bool whole = p.softmax && (bias || !p.renormalise);
  float lmax = -INFINITY;
  // Where the logits alone are compared they stay as they are: maxima pass over NaN,
  // the bounds are cut to the finite range, and so is each candidate.
  if (KEYS || whole) {
#pragma unroll
    for (int j = 0; j < N; j++) {
      l[j] = clean(l[j]);
      lmax = fmaxf(lmax, l[j]);
    }
  }

  // sum over the row's softmax (its weights unnormalised over the chosen, or its keys)
  float top = 0.0f, norm = 1.0f;
  if (whole || (KEYS && p.softmax)) top = warp_max(lmax);
  if (whole) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < N; j++) s += l[j] > kMasked ? expf(l[j] - top) : 0.0f;
    norm = warp_sum(s);
  }

  float (&f)[N] = l;  // the keys: without a bias the logits, whose order is the scores'
  float tol_s = 0.0f;  // with a bias: how far two keys' scores may be off together
  bool close = false, close_group = false;
  uint32_t keep = 0xffffffffu;
  float* s_key = nullptr;
  if constexpr (KEYS) {
    s_key = reinterpret_cast<float*>(s_dyn + (size_t)warp * E * 8);
    float smax = 0.0f;
#pragma unroll
    for (int j = 0; j < N; j++) {
      const int e = at(j);
      if (bias) {
        const float s = p.softmax ? expf(l[j] - top) / norm : 1.0f / (1.0f + expf(-l[j]));
        const bool ok = l[j] > kMasked;
        smax = fmaxf(smax, ok ? s : 0.0f);
        f[j] = ok ? fmaxf(s + __ldg(p.bias + e), -INFINITY) : -INFINITY;  // (a NaN bias: -inf)
      }
      if (e < E) s_key[e] = f[j];
    }
    // exp and the quotients are off by 2^-21.4 of a score at most; a softmax's sum by
    // one step for each addition, and its exponent's rounding weighs 2^-25 of the top score.
    // (2^-126: an exp past fp32's range makes a sigmoid below 2^-128 zero.)
    if (bias) tol_s = warp_max(smax) * (p.softmax ? (N + 16) * 0x1p-23f : 0x1p-20f) + 0x1p-126f;
    __syncwarp();
    if (p.kept < p.groups) {
      // lanes share a group's keys: sub lanes each (a power of two), merged by shuffles
      int sub = 32;
      while (sub * p.groups > 32) sub >>= 1;
      const int g = lane / sub, u = lane % sub;
      float b1 = -INFINITY, b2 = -INFINITY;
      if (g < p.groups) {
        const int n = (p.group_size + sub - 1) / sub;
        int i = g % n;  // groups start at different steps: their lanes hit different banks
        for (int q = 0; q < n; q++) {
          const int o = i * sub + u;
          if (o < p.group_size) {
            const float x = s_key[g * p.group_size + o];
            b2 = fmaxf(b2, fminf(b1, x));
            b1 = fmaxf(b1, x);
          }
          i = i + 1 == n ? 0 : i + 1;
        }
      }
      for (int d = 1; d < sub; d <<= 1) {
        const float o1 = __shfl_xor_sync(0xffffffffu, b1, d), o2 = __shfl_xor_sync(0xffffffffu, b2, d);
        b2 = fmaxf(fmaxf(b2, o2), fminf(b1, o1));
        b1 = fmaxf(b1, o1);
      }
      // a group's value: its best key (by the logit itself, exact), or the two best
      // keys' sum (softmax: without the row's common factor)
      float v = b1;
      if (p.best == 2) {
        if (bias) {
          if (b2 > -INFINITY) v += b2;
        } else if (b1 > -INFINITY) {
          const float s1 = p.softmax ? expf(b1 - top) : 1.0f / (1.0f + expf(-b1));
          const float s2 = p.softmax ? expf(b2 - top) : 1.0f / (1.0f + expf(-b2));  // 0 for none
          v = s1 + s2;
        }
      }
      int rank = 0;
      for (int o = 0; o < p.groups; o++) {
        const float x = __shfl_sync(0xffffffffu, v, o * sub);
        rank += x > v || (x == v && o < g);
      }
      const bool lead = u == 0 && g < p.groups;
      // the last kept and the first dropped group: too close to tell in fp32?
      float v0 = 0.0f, v1 = -INFINITY;
      int i0 = 0, i1 = 0;
      if (bias || p.best == 2) {
        i0 = __ffs(__ballot_sync(0xffffffffu, lead && rank == p.kept - 1)) - 1;
        i1 = __ffs(__ballot_sync(0xffffffffu, lead && rank == p.kept)) - 1;
        v0 = __shfl_sync(0xffffffffu, v, i0);
        v1 = __shfl_sync(0xffffffffu, v, i1);
      }
      // Without a bias each lane has its group's two logits: all groups again in fp64. (A
      // score is off by 2^-17.9 of itself at most, the rounding of an exponent near -104,
      // or where fp32 ends by less than 2^-128.)
      if (!bias && v1 > -INFINITY && v0 - v1 <= 0x1p-16f * v0 + 0x1p-120f) rank = group_rank64(p, b1, b2, top, g, sub);
      const uint32_t in = __ballot_sync(0xffffffffu, lead && rank < p.kept);
      keep = 0;  // groups -> bits
      for (int o = 0; o < p.groups; o++) keep |= (in >> (o * sub) & 1u) << o;
      if (bias) {
        // A value is off by its scores' errors and by the roundings of its keys and sum,
        // 2^-23 of the keys' magnitudes (not of the sum, where biases cancel). Four times
        // that: then a pair beside the border is clear when each is clear of the border's.
        const float mag = fabsf(b1) + (p.best == 2 && b2 > -INFINITY ? fabsf(b2) : 0.0f);
        const float m0 = __shfl_sync(0xffffffffu, mag, i0), m1 = __shfl_sync(0xffffffffu, mag, i1);
        auto within = [&](float hi, float lo, float m) {  // (infinite values are equal or clear)
          return lo > -INFINITY && hi < INFINITY && hi - lo <= 2.0f * tol_s + 0x1p-21f * m;
        };
        const bool pair = within(v0, v1, m0 + m1);
        // the others on both sides, which may have larger keys: when they are clear, it is
        // between these two alone
        const bool near = lead && ((rank < p.kept - 1 && within(v, v1, mag + m1)) ||
                                   (rank > p.kept && within(v0, v, m0 + mag)));
        close_group = __any_sync(0xffffffffu, near) || (pair && p.softmax);
        if (pair && !close_group) {
          const int ga = i0 / sub, gb = i1 / sub;
          keep ^= border64(p, src, ga, gb, lane) ? (1u << ga | 1u << gb) : 0u;
        }
      }
    }
    if (p.kept < p.groups) {
#pragma unroll
      for (int j = 0; j < N; j++)
        if (at(j) < E && !(keep >> group_of(p, at(j)) & 1u)) f[j] = -INFINITY;
    }
  }

  // 1. a lower bound on the K-th largest key; keys below least are not to be chosen
  const float least = bias ? -FLT_MAX : kLeast;
  float lane_max = -INFINITY;
#pragma unroll
  for (int j = 0; j < N; j++) lane_max = fmaxf(lane_max, f[j]);
  lane_max = fminf(lane_max, kLargest);
  uint32_t rest = lane_max >= least ? f32_order_key(lane_max) : 0, last = 0;
  for (int r = 0; r < K; r++) {
    const uint32_t m = warp_max_u32(rest);
    if (m == 0) break;
    last = m;
    rest = rest == m ? 0 : rest;
  }
  float bound = last ? order_key_f32(last) : least;
  if (__popc(__ballot_sync(0xffffffffu, lane_max >= bound)) < K) bound = least;  // fewer lanes than K
  // a key below the bound by less than its rounding error is a candidate too
  if (KEYS && bias) bound = fmaxf(bound - (tol_s + 0x1p-21f * fabsf(bound)), least);

  // 2. list and rank the candidates: about one in every lane that has any
  uint32_t mask = 0;
#pragma unroll
  for (int j = 0; j < N; j++) mask |= f[j] >= bound ? 1u << j : 0u;
  const int n = __popc(mask);
  int before = n;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, before, d);
    if (lane >= d) before += o;
  }
  const int count = __shfl_sync(0xffffffffu, before, 31);
  before -= n;
  int mine = -1;       // lane j: the j-th chosen expert
  float mine_l = 0.0f;
  if (count <= kCand) {
    for (; mask; mask &= mask - 1) {
      const int e = at(__ffs(mask) - 1);
      const float x = clean(to_f32(src[e]));
      s_order[warp][before] = (uint64_t)f32_order_key((bias ? s_key[e] : x) + 0.0f) << 32 | (uint32_t)~e;
      s_logit[warp][before++] = x;
    }
    __syncwarp();
    for (int c = lane; c < count; c += 32) {
      const uint64_t x = s_order[warp][c];
      int rank = 0;
      for (int o = 0; o < count; o++) rank += s_order[warp][o] > x;
      if (rank < K) s_sorted[warp][rank] = Cand{(uint32_t)(x >> 32), (int)~(uint32_t)x, s_logit[warp][c]};
    }
    __syncwarp();
    const int have = min(count, K);
    if (lane < have) {
      const Cand x = s_sorted[warp][lane];
      mine = x.e;
      mine_l = x.l;
      if constexpr (KEYS) {
        if (bias && lane + 1 < have) {
          const Cand y = s_sorted[warp][lane + 1];
          close = confusable(p, x, y, tol_s);
        }
      }
    }
    if constexpr (KEYS) {
      // the last chosen one against all that were not: behind some with its own inputs there
      // may be others
      if (bias && count > K) {
        const Cand z = s_sorted[warp][K - 1];
        const uint64_t chosen = (uint64_t)z.key << 32 | (uint32_t)~z.e;
        for (int c = lane; c < count; c += 32) {
          const uint64_t x = s_order[warp][c];
          if (x < chosen) close |= confusable(p, z, Cand{(uint32_t)(x >> 32), (int)~(uint32_t)x, s_logit[warp][c]}, tol_s);
        }
      }
      if (__any_sync(0xffffffffu, close) && !p.softmax && count <= 32) {
        // the candidates' keys in fp64, ranked again, one lane each
        close = false;
        double* s64 = reinterpret_cast<double*>(s_key);
        double k64 = 0.0;
        Cand x = {};
        __syncwarp();
        if (lane < count) {
          x = Cand{0, (int)~(uint32_t)s_order[warp][lane], s_logit[warp][lane]};
          k64 = sigmoid64((double)x.l) + (double)__ldg(p.bias + x.e);
          s64[lane] = k64;
        }
        __syncwarp();
        if (lane < count) {
          int rank = 0;
          for (int o = 0; o < count; o++) rank += s64[o] > k64 || (s64[o] == k64 && (int)~(uint32_t)s_order[warp][o] < x.e);
          if (rank < K) s_sorted[warp][rank] = x;
        }
        __syncwarp();
        if (lane < have) {
          mine = s_sorted[warp][lane].e;
          mine_l = s_sorted[warp][lane].l;
        }
      }
    }
  } else {
    if (bias) close = true;  // too many to rank: decide them in fp64
    else mine = choose_rounds<T>(p, src, keep, lane);
    if (mine >= 0) mine_l = clean(to_f32(src[mine]));
  }
  if constexpr (KEYS) {
    if (__any_sync(0xffffffffu, close || close_group)) {
      __syncwarp();
      mine = choose64<T>(p, src, reinterpret_cast<double*>(s_key), lane);
      mine_l = mine >= 0 ? clean(to_f32(src[mine])) : 0.0f;
    }
  }

  // weights
  const bool there = lane < K && mine >= 0;
  float s;
  // (a renormalised row's common factor, exp of its largest chosen logit, is taken out before
  // fp32 loses it: a bias may choose experts whose scores are far below the row's largest)
  if (p.softmax) {
    // (without keys `whole` says the same; asking for it again: 65536 rows 41 us, not 39)
    const float m = (KEYS ? !p.renormalise : whole) ? top : warp_max(there ? mine_l : -INFINITY);
    s = there ? expf(mine_l - m) : 0.0f;
    if (!p.renormalise) s /= norm;
  } else {
    // exp(l) / (1 + exp(l)) below 0: the other form's exp would overflow
    const float m = p.renormalise ? fminf(warp_max(there ? mine_l : -INFINITY), 0.0f) : 0.0f;
    s = there ? (mine_l < 0.0f ? expf(mine_l - m) : 1.0f) / (1.0f + expf(-fabsf(mine_l))) : 0.0f;
  }
  if (p.renormalise) {
    const float sum = warp_sum(s);
    s = sum > 0.0f ? s / sum : 0.0f;
  }
  if (lane < K) {
    p.idx[row * K + lane] = there ? mine : -1;
    p.w[row * K + lane] = there ? p.scale * s : 0.0f;
  }
}

template <typename T, int N, bool VEC>
cudaError_t launch_n(const RouteParams& p, bool keys, cudaStream_t s) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)((p.rows + kWarps - 1) / kWarps));
  c.blockDim = dim3(kWarps * 32);
  c.dynamicSmemBytes = keys ? (size_t)kWarps * p.E * 8 : 0;  // at most 32 KB (E = 1024)
  c.stream = s;
  return keys ? cudaLaunchKernelEx(&c, route_kernel<T, N, VEC, true>, p)
              : cudaLaunchKernelEx(&c, route_kernel<T, N, VEC, false>, p);
}

template <typename T>
cudaError_t launch_t(const RouteParams& p, bool keys, cudaStream_t s) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p.logits);
  // four consecutive logits in one load: every row starts on a multiple of it
  const bool vec = p.E % 4 == 0 && p.stride % 4 == 0 && a % (4 * sizeof(T)) == 0 && p.E > 64;
  if (vec) {
    if (p.E <= 128) return launch_n<T, 4, true>(p, keys, s);
    if (p.E <= 256) return launch_n<T, 8, true>(p, keys, s);
    if (p.E <= 512) return launch_n<T, 16, true>(p, keys, s);
    return launch_n<T, 32, true>(p, keys, s);
  }
  if (p.E <= 64) return launch_n<T, 2, false>(p, keys, s);
  if (p.E <= 128) return launch_n<T, 4, false>(p, keys, s);
  if (p.E <= 256) return launch_n<T, 8, false>(p, keys, s);
  if (p.E <= 512) return launch_n<T, 16, false>(p, keys, s);
  return launch_n<T, 32, false>(p, keys, s);
}

}  // namespace

cudaError_t launch_route(const moe_route_config& c, const void* logits, int64_t stride, const float* bias,
                         int64_t rows, int32_t* idx, float* w, cudaStream_t s) {
  RouteParams p;
  p.logits = logits;
  p.stride = stride;
  p.bias = bias;
  p.rows = rows;
  p.idx = idx;
  p.w = w;
  p.E = c.num_experts;
  p.K = c.top_k;
  p.softmax = c.score == MOE_ROUTE_SOFTMAX;
  p.groups = c.num_groups;
  p.kept = c.top_groups;
  p.best = c.group_best;
  p.group_size = c.num_experts / c.num_groups;
  p.group_magic = p.group_size > 1 ? 0xffffffffu / p.group_size + 1 : 0;
  p.renormalise = c.renormalise != 0;
  p.scale = c.scale;
  const bool keys = bias || c.top_groups < c.num_groups;
  return c.logits_dtype == MOE_F32 ? launch_t<float>(p, keys, s) : launch_t<__nv_bfloat16>(p, keys, s);
}

}  // namespace rows
}  // namespace moe
