// Rotary positions of new tokens and the write of keys and values into the paged cache.
//
//   x' = m (x cos t - y sin t),  y' = m (y cos t + x sin t),  t = position * f_j
//
// for the pairs (x, y) = (j, j + r/2) (half layout) or (2j, 2j + 1) (interleaved) of the first r
// values of a head.  f_j comes as the fraction of a turn per position, scaled by 2^64, so the phase
// is one 64-bit product: whole turns fall out by the wrap.  The frequencies are rounded from 64-bit floating
// point, which at a position of 10^6 leaves the phase exact to 2^-35 of a turn, where an fp32 product would
// have lost all but four bits of it.
#include "spec_device.cuh"
#include "step_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace sv {

namespace {

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

// Any size, alignment and stride: one CTA per token: the token's request and cache slot, its r/2 angles in shared
// memory, then every head's values, 1 pair (or 1 value behind the rotated part) per thread and step.
template <int DTYPE>
__global__ void __launch_bounds__(kRopeThreads) rope_scalar_kernel(const RopeParams p) {
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


constexpr int kRopeMaxTokens = 8;   // tokens per CTA: one warp each finds the request and the slot

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

// 16-byte pieces of VEC values; V of a token's pieces are pairs of pieces (half layout), single
// pieces of pairs (interleaved), or copies.
template <int DTYPE>
struct Piece {
  using T = typename RopeType<DTYPE>::T;
  static constexpr int VEC = 16 / sizeof(T);
  uint4 raw;
  __device__ __forceinline__ void load(const T* p) { raw = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<uint4*>(p) = raw; }
  __device__ __forceinline__ float get(int i) const { return to_f(reinterpret_cast<const T*>(&raw)[i]); }
  __device__ __forceinline__ void put(int i, float x) { from_f(x, reinterpret_cast<T*>(&raw) + i); }
};

// The fast form: heads, halves and strides are whole 16-byte pieces.  A CTA takes `per_cta` tokens:
// a warp each looks up the request, position and cache slot; the CTA computes the tokens' angles once
// for all heads; then each thread moves 16-byte pieces (a piece and its partner in the half layout),
// the next pieces' loads issued ahead of the current ones' stores.
// Bound: HBM (2 x (q + k + v) bytes, no reuse).
template <int DTYPE, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p, int per_cta) {
  using T = typename RopeType<DTYPE>::T;
  using Pc = Piece<DTYPE>;
  constexpr int VEC = Pc::VEC, PP = INTERLEAVED ? VEC / 2 : VEC;   // values of a piece, pairs of a unit
  extern __shared__ __align__(16) float2 s_cs[];   // [per_cta][rotary / 2]
  __shared__ long long s_k[kRopeMaxTokens], s_v[kRopeMaxTokens];
  __shared__ int s_pos[kRopeMaxTokens], s_req[kRopeMaxTokens];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n0 = blockIdx.x * per_cta, tokens = min(per_cta, p.c.N - n0);
  const int half = p.rotary / 2, D = p.c.D, Hk = p.c.Hkv;
  const int turn = (INTERLEAVED ? p.rotary : half) / VEC;   // rotated units per head
  const int per_head = turn + (D - p.rotary) / VEC;
  const int rot_units = (p.Hq + Hk) * per_head;
  const int units = rot_units + (p.c.k ? Hk * (D / VEC) : 0);   // per token
  const int total = tokens * units;
  // quotients of small numbers by the sizes above: floor(n ceil(2^32 / d) / 2^32) is exact while n d < 2^32.
  // d < 2^16 (the launch sees to it) and n < 2^16: several tokens have 2048 pieces together, one fewer than
  // 2^16.  Sizes of 1 wrap to 0 and are handled apart.
  auto inverse = [](int d) { return d > 1 ? 0xffffffffu / static_cast<unsigned>(d) + 1u : 0u; };
  const unsigned inv_units = inverse(units), inv_head = inverse(per_head), inv_value = inverse(D / VEC);
  auto quotient = [](int n, unsigned inv) { return inv ? static_cast<int>(__umulhi(static_cast<unsigned>(n), inv)) : n; };
  // strides fit 32 bits here: one wide multiplication per address
  const int q_token = static_cast<int>(p.q_token), k_token = static_cast<int>(p.k_token), v_token = static_cast<int>(p.v_token);
  const int q_head = static_cast<int>(p.q_head), k_head = static_cast<int>(p.k_head), v_head = static_cast<int>(p.v_head);
  const int qo_token = static_cast<int>(p.qo_token), ko_token = static_cast<int>(p.ko_token);
  const int qo_head = static_cast<int>(p.qo_head), ko_head = static_cast<int>(p.ko_head);
  const int kc_head = static_cast<int>(p.c.k_head), vc_head = static_cast<int>(p.c.v_head);
  auto at2 = [](int i, int si, int j, int sj) { return static_cast<long long>(i) * si + static_cast<long long>(j) * sj; };

  struct Unit {
    Pc a, b;
    T *d0, *d1;
    int t, kind, at;   // kind 0: rotate, 1: copy
  };
  auto load = [&](int u, Unit& x) {
    x.t = quotient(u, inv_units);
    int r = u - x.t * units;
    const int n = n0 + x.t;
    const T* src;
    if (r < rot_units) {
      const int h = quotient(r, inv_head), j = r - h * per_head, hk = h - p.Hq;
      x.kind = j < turn ? 0 : 1;
      x.at = j < turn ? j * VEC : p.rotary + (j - turn) * VEC;
      src = hk < 0 ? reinterpret_cast<const T*>(p.q) + at2(n, q_token, h, q_head)
                   : reinterpret_cast<const T*>(p.k) + at2(n, k_token, hk, k_head);
      x.d0 = hk < 0 ? reinterpret_cast<T*>(p.q_out) + at2(n, qo_token, h, qo_head)
                    : (p.k_out ? reinterpret_cast<T*>(p.k_out) + at2(n, ko_token, hk, ko_head) : nullptr);
      x.d1 = hk < 0 || !p.c.k ? nullptr : reinterpret_cast<T*>(p.c.k) + at2(hk, kc_head, 0, 0);
      x.a.load(src + x.at);
      if (!INTERLEAVED && x.kind == 0) x.b.load(src + x.at + half);
    } else {
      r -= rot_units;
      const int h = quotient(r, inv_value), j = r - h * (D / VEC);
      x.kind = 2;
      x.at = j * VEC;
      x.d0 = nullptr;
      x.d1 = reinterpret_cast<T*>(p.c.v) + at2(h, vc_head, 0, 0);
      x.a.load(reinterpret_cast<const T*>(p.v) + at2(n, v_token, h, v_head) + x.at);
    }
  };
  Unit cur;
  int u = tid;
  if (u < total) load(u, cur);   // in flight while the tokens' slots are looked up

  for (int t = warp; t < tokens; t += kRopeThreads / 32) {
    const int n = n0 + t, b = request_of(p.c.cu_q, p.c.B, n, lane);
    if (lane == 0) {
      long long ks = -1, vs = -1;
      int pos = 0;
      const bool has = b >= 0 && b < p.c.B;
      if (has) {
        pos = __ldg(p.c.kv_lens + b) - (__ldg(p.c.cu_q + b + 1) - n);
        if (p.c.k && pos >= 0) {
          const int col = pos / p.c.page_size, in = pos % p.c.page_size;
          const int pg = col < p.c.table_width ? __ldg(p.c.table + b * p.c.table_stride + col) : -1;
          if (pg < 0 || pg >= p.c.pages) {
            atomicOr(p.status, kStatusPageRange);
          } else {
            ks = pg * p.c.k_page + in * p.c.k_token;
            vs = pg * p.c.v_page + in * p.c.v_token;
          }
        }
      }
      s_k[t] = ks;
      s_v[t] = vs;
      s_pos[t] = pos;
      s_req[t] = has;
    }
  }
  __syncthreads();
  for (int i = tid; i < tokens * half; i += kRopeThreads) {
    const int t = i / half;
    const float2 c = phase_cs(p.freq[i - t * half] * static_cast<unsigned long long>(static_cast<long long>(s_pos[t])));
    // two pairs' angles together, then the units side by side: the lanes' 16-byte reads fall on distinct banks
    const int j = i - t * half, e = j & (PP - 1);
    s_cs[t * half + ((e >> 1) * turn + j / PP) * 2 + (e & 1)] = make_float2(c.x * p.factor, c.y * p.factor);
  }
  __syncthreads();
  while (u < total) {
    Unit next;
    const int un = u + kRopeThreads;
    if (un < total) load(un, next);
    if (s_req[cur.t]) {
      if (cur.kind == 0) {
        const float4* cs = reinterpret_cast<const float4*>(s_cs + cur.t * half) + cur.at / VEC;
#pragma unroll
        for (int i = 0; i < PP; i += 2) {
          const float4 w = cs[(i >> 1) * turn];   // cos, sin of pairs i and i + 1
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float c = e ? w.z : w.x, s = e ? w.w : w.y;
            if (INTERLEAVED) {
              const float x = cur.a.get(2 * (i + e)), y = cur.a.get(2 * (i + e) + 1);
              cur.a.put(2 * (i + e), x * c - y * s);
              cur.a.put(2 * (i + e) + 1, y * c + x * s);
            } else {
              const float x = cur.a.get(i + e), y = cur.b.get(i + e);
              cur.a.put(i + e, x * c - y * s);
              cur.b.put(i + e, y * c + x * s);
            }
          }
        }
      }
      const long long slot = cur.kind == 2 ? s_v[cur.t] : s_k[cur.t];
      const bool pair = !INTERLEAVED && cur.kind == 0;
      if (cur.d0) {
        cur.a.store(cur.d0 + cur.at);
        if (pair) cur.b.store(cur.d0 + cur.at + half);
      }
      if (cur.d1 && slot >= 0) {
        cur.a.store(cur.d1 + slot + cur.at);
        if (pair) cur.b.store(cur.d1 + slot + cur.at + half);
      }
    }
    cur = next;
    u = un;
  }
}

}  // namespace

cudaError_t launch_rope(int dtype, const RopeParams& p, int sms, cudaStream_t stream) {
  const int vec = dtype == 0 ? 4 : 8;
  // whole 16-byte pieces: sizes, strides and bases
  const long long strides[] = {p.q_token, p.q_head, p.k_token, p.k_head, p.qo_token, p.qo_head,
                               p.k_out ? p.ko_token : 0, p.k_out ? p.ko_head : 0, p.c.k ? p.v_token : 0, p.c.k ? p.v_head : 0};
  bool whole = p.c.D % vec == 0 && p.rotary % (p.interleaved ? vec : 2 * vec) == 0;
  for (long long s : strides) whole = whole && s % vec == 0 && s >= 0 && s < (1ll << 31);
  whole = whole && p.c.k_head < (1ll << 31) && p.c.v_head < (1ll << 31);
  // the piece kernel's 32-bit quotients (above) hold up to 65,535 pieces a token
  const long long units = (p.Hq + 2ll * p.c.Hkv) * (p.c.D / vec);
  whole = whole && units < (1 << 16);
  const void* bases[] = {p.q, p.k, p.c.k ? p.v : nullptr, p.q_out, p.k_out};
  for (const void* b : bases) whole = whole && (reinterpret_cast<uintptr_t>(b) & 15) == 0;
  if (!whole) {
    const dim3 grid(p.c.N), block(kRopeThreads);
    const size_t smem = sizeof(float2) * (p.rotary / 2);
    if (dtype == 0) rope_scalar_kernel<0><<<grid, block, smem, stream>>>(p);
    if (dtype == 1) rope_scalar_kernel<1><<<grid, block, smem, stream>>>(p);
    if (dtype == 2) rope_scalar_kernel<2><<<grid, block, smem, stream>>>(p);
    return cudaGetLastError();
  }
  // few tokens: a CTA each; many: as many tokens a CTA as make about 2048 pieces.  40 + 8 heads of 128, bf16, on
  // the device, a CTA a token against 2048 pieces: 304 tokens 4.7 : 5.5 us, 608 (four an SM) 7.1 : 8.4, 1088
  // 9.2 : 10.4, 2048 13.8 : 13.2; so the rule changes over early rather than late.  8192 tokens (201 MB) take
  // 39 us (5.2 TB/s, 76 % of measured HBM); with quotients by division 41, then 43 with 1024 pieces, 49 with
  // 4096, 45 with 256 threads, 47 with four pieces in flight a thread instead of two.
  int per = p.c.N <= 4 * sms ? 1 : static_cast<int>(2048 / (units > 0 ? units : 1));
  per = per < 1 ? 1 : per > kRopeMaxTokens ? kRopeMaxTokens : per;
  const dim3 grid((p.c.N + per - 1) / per), block(kRopeThreads);
  const size_t smem = sizeof(float2) * (p.rotary / 2) * per;
  const int kind = dtype * 2 + (p.interleaved ? 1 : 0);
  if (kind == 0) rope_kernel<0, false><<<grid, block, smem, stream>>>(p, per);
  if (kind == 1) rope_kernel<0, true><<<grid, block, smem, stream>>>(p, per);
  if (kind == 2) rope_kernel<1, false><<<grid, block, smem, stream>>>(p, per);
  if (kind == 3) rope_kernel<1, true><<<grid, block, smem, stream>>>(p, per);
  if (kind == 4) rope_kernel<2, false><<<grid, block, smem, stream>>>(p, per);
  if (kind == 5) rope_kernel<2, true><<<grid, block, smem, stream>>>(p, per);
  return cudaGetLastError();
}

}  // namespace sv
