// What the kernels that write new tokens into a paged cache share: their types, rotary phases, the request of a token.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "spec_device.cuh"
#include "step_internal.h"

namespace sv {

constexpr int kRopeThreads = 128;

template <int DTYPE>
struct RopeType;
template <>
struct RopeType<0> {
  using T = float;
};
template <>
struct RopeType<1> {
  using T = __nv_bfloat16;
};
template <>
struct RopeType<2> {
  using T = __half;
};
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f(float x, float* y) { *y = x; }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16* y) { *y = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f(float x, __half* y) { *y = __float2half_rn(x); }

// cos and sin of 2 pi phase / 2^64.
__device__ __forceinline__ float2 phase_cs(unsigned long long phase) {
  const float half_turns = static_cast<float>(static_cast<int>(phase >> 32)) * 4.656612873077393e-10f;   // 2^-31
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c, s);
}

// Largest b with cu[b] <= n, by a 32-way search of one warp (-1: none).
__device__ __forceinline__ int request_of(const int32_t* cu, int B, int n, int lane) {
  int lo = -1, hi = B + 1;   // cu[lo] <= n < cu[hi], with cu[-1] = -inf and cu[B + 1] = +inf
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
    const bool le = at < hi && __ldg(cu + at) <= n;
    const int k = __popc(__ballot_sync(0xffffffffu, le));
    const int nlo = lo + k * step;
    hi = min(hi, nlo + step);
    lo = nlo;
  }
  return lo;
}

}  // namespace sv
