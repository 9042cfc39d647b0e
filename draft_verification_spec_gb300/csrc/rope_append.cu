// Rotary positions of new tokens and the write of keys and values into the paged cache.
//
//   x' = m (x cos t - y sin t),  y' = m (y cos t + x sin t),  t = position * f_j
//
// for the pairs (x, y) = (j, j + r/2) (half layout) or (2j, 2j + 1) (interleaved) of the first r
// values of a head.  f_j comes as the fraction of a turn per position, scaled by 2^64, so the phase
// is one 64-bit product: whole turns fall out by the wrap, and a position of 10^6 keeps the phase
// to 2^-44 of a turn where an fp32 product would have lost all but four bits of it.
#include "spec_device.cuh"
#include "step_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace sv {

namespace {

constexpr int kRopeThreads = 256;

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

// One CTA per token: the token's request and cache slot, its r/2 angles in shared memory, then every
// head's values, 1 pair (or 1 value behind the rotated part) per thread and step.
template <int DTYPE>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  using T = typename RopeType<DTYPE>::T;
  extern __shared__ float2 cs[];   // [rotary / 2]
  __shared__ int s_b;
  __shared__ long long s_slot[2];
  const int n = blockIdx.x, tid = threadIdx.x;
  if (tid == 0) s_b = -1;
  __syncthreads();
  for (int b = tid; b < p.c.B; b += kRopeThreads)
    if (__ldg(p.c.cu_q + b) <= n && n < __ldg(p.c.cu_q + b + 1)) s_b = b;
  __syncthreads();
  const int b = s_b;
  if (b < 0) return;   // a token of no request
  const int pos = __ldg(p.c.kv_lens + b) - (__ldg(p.c.cu_q + b + 1) - n);
  if (tid == 0) {
    s_slot[0] = s_slot[1] = -1;
    if (p.c.k) {
      const int col = pos / p.c.page_size, in = pos % p.c.page_size;
      const int pg = pos >= 0 && col < p.c.table_width ? __ldg(p.c.table + b * p.c.table_stride + col) : -1;
      if (pos >= 0 && (pg < 0 || pg >= p.c.pages)) atomicOr(p.status, kStatusPageRange);
      if (pg >= 0 && pg < p.c.pages) {
        s_slot[0] = pg * p.c.k_page + in * p.c.k_token;
        s_slot[1] = pg * p.c.v_page + in * p.c.v_token;
      }
    }
  }
  const int half = p.rotary / 2;
  for (int j = tid; j < half; j += kRopeThreads) {
    float2 c = phase_cs(p.freq[j] * static_cast<unsigned long long>(static_cast<long long>(pos)));
    cs[j] = make_float2(c.x * p.factor, c.y * p.factor);
  }
  __syncthreads();
  const int D = p.c.D, rest = D - p.rotary, per = half + rest;
  const T* q = reinterpret_cast<const T*>(p.q) + n * p.q_token;
  const T* k = reinterpret_cast<const T*>(p.k) + n * p.k_token;
  const T* v = reinterpret_cast<const T*>(p.v) + n * p.v_token;
  T* qo = reinterpret_cast<T*>(p.q_out) + n * p.qo_token;
  T* ko = p.k_out ? reinterpret_cast<T*>(p.k_out) + n * p.ko_token : nullptr;
  T* kc = s_slot[0] >= 0 ? reinterpret_cast<T*>(p.c.k) + s_slot[0] : nullptr;
  T* vc = s_slot[1] >= 0 ? reinterpret_cast<T*>(p.c.v) + s_slot[1] : nullptr;
  for (int id = tid; id < (p.Hq + p.c.Hkv) * per; id += kRopeThreads) {
    const int h = id / per, j = id % per, hk = h - p.Hq;
    const T* src = hk < 0 ? q + h * p.q_head : k + hk * p.k_head;
    T* d0 = hk < 0 ? qo + h * p.qo_head : (ko ? ko + hk * p.ko_head : nullptr);
    T* d1 = hk < 0 || !kc ? nullptr : kc + hk * p.c.k_head;
    if (j < half) {
      const int ia = p.interleaved ? 2 * j : j, ib = p.interleaved ? 2 * j + 1 : j + half;
      const float x = to_f(src[ia]), y = to_f(src[ib]);
      const float2 c = cs[j];
      T a, e;
      from_f(x * c.x - y * c.y, &a);
      from_f(y * c.x + x * c.y, &e);
      if (d0) d0[ia] = a, d0[ib] = e;
      if (d1) d1[ia] = a, d1[ib] = e;
    } else {
      const int i = p.rotary + j - half;
      const T x = src[i];
      if (d0) d0[i] = x;
      if (d1) d1[i] = x;
    }
  }
  if (vc)
    for (int id = tid; id < p.c.Hkv * D; id += kRopeThreads) {
      const int h = id / D, i = id % D;
      vc[h * p.c.v_head + i] = v[h * p.v_head + i];
    }
}

}  // namespace

cudaError_t launch_rope(int dtype, const RopeParams& p, cudaStream_t stream) {
  const dim3 grid(p.c.N), block(kRopeThreads);
  const size_t smem = sizeof(float2) * (p.rotary / 2);
  if (dtype == 0) rope_kernel<0><<<grid, block, smem, stream>>>(p);
  if (dtype == 1) rope_kernel<1><<<grid, block, smem, stream>>>(p);
  if (dtype == 2) rope_kernel<2><<<grid, block, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace sv
