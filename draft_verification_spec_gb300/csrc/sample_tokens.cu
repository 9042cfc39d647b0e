// Sampling with temperature, top-k, top-p and min-p from given uniforms.
//
// A row's tokens are taken in the order (logit descending, index ascending).  With weights
// w = 2^((z - max) c), c = log2(e) / T, each filter keeps a prefix of that order:
//   top-k   the first k;
//   top-p   of those, the shortest prefix whose weight reaches top_p x the weight of the k;
//   min-p   the tokens with w >= min_p (the largest w is 1);
// the kept ones are the first n = min of the three (at least one), and the drawn token is the first
// whose inclusive prefix weight is strictly above u x the weight of the n.
//
// Every question is "which element of the order does a count or a weight reach", answered by a
// descent over the digits of the logits' ordered keys: a histogram of counts and weights per digit,
// then the digit that the target falls in, then the next one among the elements that match so far.
// Equal logits are told apart by their index at the end.
#include <cuda_bf16.h>

#include "sample_weight.cuh"
#include "step_internal.h"

namespace sv {

namespace {

constexpr int kThreads = 1024;
constexpr int kDigitBits = 11, kBins = 1 << kDigitBits;

template <int DTYPE>
__device__ __forceinline__ float row_logit(const void* row, int i) {
  if (DTYPE == 1) return __uint_as_float(static_cast<unsigned>(__ldg(static_cast<const uint16_t*>(row) + i)) << 16);
  return __ldg(static_cast<const float*>(row) + i);
}
// Ordered key; NaN counts as -inf, which is never drawn.
__device__ __forceinline__ uint32_t sample_key(float z) { return ord_key(z != z ? ninf() : z); }
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

struct Prefix {
  unsigned cnt;            // elements before the group in the order
  unsigned long long mass;
  uint32_t key;            // the group's key
};

struct Smem {
  unsigned long long tab[64];
  unsigned cnt[kBins], lo[kBins], hi[kBins];
  unsigned wcnt[32];
  unsigned long long wmass[32];
  float wmax[32];
  Prefix found;
  int token;
};

// Block-wide: the group of equal keys in which the order's count (BY_COUNT) or weight reaches `target`
// (1 <= target <= the row's).
template <int DTYPE, bool BY_COUNT>
__device__ Prefix descend(const void* row, int V, const WeightScale& ws, unsigned long long target, Smem& s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Prefix at = {0u, 0ull, 0u};
  int bits = DTYPE == 1 ? 16 : 32;     // key bits still to be fixed
  uint32_t fixed = 0;                  // the digits found so far, right-aligned
  while (bits > 0) {
    const int digit = bits < kDigitBits ? bits : kDigitBits;
    bits -= digit;
    for (int i = tid; i < kBins; i += kThreads) s.cnt[i] = s.lo[i] = s.hi[i] = 0u;
    __syncthreads();
    for (int i = tid; i < V; i += kThreads) {
      const float z = row_logit<DTYPE>(row, i);
      uint32_t key = sample_key(z);
      if (DTYPE == 1) key >>= 16;
      if ((static_cast<unsigned long long>(key) >> (bits + digit)) != fixed || !(z > ninf())) continue;
      const unsigned d = (key >> bits) & ((1u << digit) - 1u);
      const unsigned long long w = weight_of(z, ws, s.tab);
      atomicAdd(&s.cnt[d], 1u);
      const unsigned lo = static_cast<unsigned>(w);
      const unsigned old = atomicAdd(&s.lo[d], lo);
      const unsigned up = static_cast<unsigned>(w >> 32) + (old + lo < old ? 1u : 0u);
      if (up) atomicAdd(&s.hi[d], up);
    }
    __syncthreads();
    // thread t holds the bins 2t, 2t + 1 from the top; a block scan gives what lies before them
    unsigned c[2];
    unsigned long long m[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int bin = kBins - 1 - (2 * tid + e);
      c[e] = s.cnt[bin];
      m[e] = (static_cast<unsigned long long>(s.hi[bin]) << 32) + s.lo[bin];
    }
    unsigned ic = c[0] + c[1];
    unsigned long long im = m[0] + m[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned tc = __shfl_up_sync(0xffffffffu, ic, o);
      const unsigned long long tm = __shfl_up_sync(0xffffffffu, im, o);
      if (lane >= o) ic += tc, im += tm;
    }
    if (lane == 31) s.wcnt[warp] = ic, s.wmass[warp] = im;
    __syncthreads();
    for (int k = 0; k < warp; ++k) ic += s.wcnt[k], im += s.wmass[k];
    unsigned bc = at.cnt + ic - c[0] - c[1];
    unsigned long long bm = at.mass + im - m[0] - m[1];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const bool before = BY_COUNT ? bc < target : bm < target;
      const bool reached = BY_COUNT ? bc + c[e] >= target : bm + m[e] >= target;
      if (before && reached) s.found = {bc, bm, static_cast<uint32_t>((fixed << digit) | (kBins - 1 - (2 * tid + e)))};
      bc += c[e];
      bm += m[e];
    }
    __syncthreads();
    at = s.found;
    fixed = at.key;
    __syncthreads();
  }
  return at;
}

// Block-wide sum of a count and a weight.
__device__ void block_sum(unsigned& c, unsigned long long& m, Smem& s) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    c += __shfl_xor_sync(0xffffffffu, c, o);
    m += __shfl_xor_sync(0xffffffffu, m, o);
  }
  if ((threadIdx.x & 31) == 0) s.wcnt[threadIdx.x / 32] = c, s.wmass[threadIdx.x / 32] = m;
  __syncthreads();
  c = 0;
  m = 0;
  for (int k = 0; k < kThreads / 32; ++k) c += s.wcnt[k], m += s.wmass[k];
  __syncthreads();
}

template <int DTYPE>
__global__ void __launch_bounds__(kThreads) sample_kernel_row(const SampleParams p) {
  extern __shared__ __align__(16) uint8_t raw[];
  Smem& s = *reinterpret_cast<Smem*>(raw);
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, V = p.V;
  const int esz = DTYPE == 1 ? 2 : 4;
  const void* row = static_cast<const uint8_t*>(p.logits) + static_cast<long long>(r) * p.stride * esz;
  if (tid < 64) s.tab[tid] = kExp2Table[tid];
  // the row's largest logit
  float mx = ninf();
  for (int i = tid; i < V; i += kThreads) mx = fmaxf(mx, row_logit<DTYPE>(row, i));
  mx = warp_max(mx);
  if (lane == 0) s.wmax[tid / 32] = mx;
  __syncthreads();
  mx = warp_max(s.wmax[lane]);
  __syncthreads();

  float T = p.temperature ? p.temperature[r] : p.temperature0;
  int k = p.top_k ? p.top_k[r] : p.top_k0;
  const float top_p = p.top_p ? p.top_p[r] : p.top_p0, min_p = p.min_p ? p.min_p[r] : p.min_p0;
  if (!(T > 0.f)) {   // greedy: the first of the order
    T = 1.f;
    k = 1;
  }
  const WeightScale ws = weight_scale(mx, T);
  const unsigned long long least = min_p > 0.f ? static_cast<unsigned long long>(ceil(static_cast<double>(min_p) * kWeightOne)) : 0ull;

  // finite tokens and their weight; those of at least min_p
  unsigned n_all = 0, n_min = 0;
  unsigned long long m_all = 0, m_min = 0;
  for (int i = tid; i < V; i += kThreads) {
    const float z = row_logit<DTYPE>(row, i);
    if (!(z > ninf())) continue;
    const unsigned long long w = weight_of(z, ws, s.tab);
    ++n_all;
    m_all += w;
    if (w >= least) ++n_min, m_min += w;
  }
  block_sum(n_all, m_all, s);
  block_sum(n_min, m_min, s);

  unsigned n = 0;
  unsigned long long mass = 0;
  int token = -1;
  float prob = 0.f;
  Prefix cut = {0u, 0ull, 0u};
  if (n_all > 0) {
    n = n_all;
    mass = m_all;
    if (k > 0 && static_cast<unsigned>(k) < n) {
      const Prefix g = descend<DTYPE, true>(row, V, ws, k, s);
      n = k;
      mass = g.mass + (k - g.cnt) * weight_of(key_logit(DTYPE == 1 ? g.key << 16 | (g.key & 0x8000u ? 0u : 0xffffu) : g.key), ws, s.tab);
    }
    if (top_p < 1.f) {
      const double goal = ceil(fmax(static_cast<double>(top_p), 0.0) * static_cast<double>(mass));
      unsigned long long target = goal < 1.0 ? 1ull : static_cast<unsigned long long>(goal);
      if (target > mass) target = mass;
      const Prefix g = descend<DTYPE, false>(row, V, ws, target, s);
      const unsigned long long w = weight_of(key_logit(DTYPE == 1 ? g.key << 16 | (g.key & 0x8000u ? 0u : 0xffffu) : g.key), ws, s.tab);
      const unsigned in = static_cast<unsigned>((target - g.mass + w - 1) / w);
      if (g.cnt + in < n) n = g.cnt + in, mass = g.mass + in * w;
    }
    if (min_p > 0.f && n_min < n) {
      n = n_min > 0 ? n_min : 1;
      mass = n_min > 0 ? m_min : kWeightOne;
    }
    // the draw
    const float u = p.uniforms[r];
    const double td = u > 0.f ? floor(static_cast<double>(u) * static_cast<double>(mass)) : 0.0;
    unsigned long long t = td >= static_cast<double>(mass) ? mass - 1 : static_cast<unsigned long long>(td);
    if (t >= mass) t = mass - 1;
    const Prefix g = descend<DTYPE, false>(row, V, ws, t + 1, s);
    const float z = key_logit(DTYPE == 1 ? g.key << 16 | (g.key & 0x8000u ? 0u : 0xffffu) : g.key);
    const unsigned long long w = weight_of(z, ws, s.tab);
    unsigned rank = static_cast<unsigned>((t + 1 - g.mass + w - 1) / w) - 1;   // among the equal ones
    prob = static_cast<float>(static_cast<double>(w) / static_cast<double>(mass));
    if (p.filtered) cut = descend<DTYPE, true>(row, V, ws, n, s);
    // the rank-th token with that logit: contiguous shares, a scan of their counts
    const int share = (V + kThreads - 1) / kThreads, i0 = min(V, tid * share), i1 = min(V, i0 + share);
    unsigned mine = 0, eq_cut = 0;
    const float zc = p.filtered ? key_logit(DTYPE == 1 ? cut.key << 16 | (cut.key & 0x8000u ? 0u : 0xffffu) : cut.key) : 0.f;
    for (int i = i0; i < i1; ++i) {
      const float x = row_logit<DTYPE>(row, i);
      mine += x == z;
      eq_cut += x == zc;
    }
    unsigned a = mine, e = eq_cut;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned ta = __shfl_up_sync(0xffffffffu, a, o), te = __shfl_up_sync(0xffffffffu, e, o);
      if (lane >= o) a += ta, e += te;
    }
    if (lane == 31) s.cnt[tid / 32] = a, s.lo[tid / 32] = e;
    __syncthreads();
    for (int q = 0; q < tid / 32; ++q) a += s.cnt[q], e += s.lo[q];
    a -= mine;
    e -= eq_cut;
    if (rank >= a && rank < a + mine) {
      unsigned left = rank - a;
      for (int i = i0; i < i1; ++i)
        if (row_logit<DTYPE>(row, i) == z && left-- == 0) {
          s.token = i;
          break;
        }
    }
    if (p.filtered) {
      const unsigned keep_eq = n - cut.cnt;   // of the tokens equal to the cut's logit
      for (int i = i0; i < i1; ++i) {
        const float x = row_logit<DTYPE>(row, i);
        const bool keep = x > zc || (x == zc && e < keep_eq);
        e += x == zc;
        const long long at = static_cast<long long>(r) * p.filtered_stride + i;
        if (DTYPE == 1)
          static_cast<uint16_t*>(p.filtered)[at] = keep ? static_cast<const uint16_t*>(row)[i] : 0xff80u;
        else
          static_cast<float*>(p.filtered)[at] = keep ? static_cast<const float*>(row)[i] : ninf();
      }
    }
    __syncthreads();
    token = s.token;
  } else if (p.filtered) {
    for (int i = tid; i < V; i += kThreads) {
      const long long at = static_cast<long long>(r) * p.filtered_stride + i;
      if (DTYPE == 1)
        static_cast<uint16_t*>(p.filtered)[at] = 0xff80u;
      else
        static_cast<float*>(p.filtered)[at] = ninf();
    }
  }
  if (tid == 0) {
    p.tokens[r] = token;
    if (p.probs) p.probs[r] = prob;
    if (p.kept) p.kept[r] = static_cast<int32_t>(n);
  }
}

}  // namespace

cudaError_t launch_sample(int dtype, const SampleParams& p, cudaStream_t stream) {
  const void* fn = dtype == 1 ? reinterpret_cast<const void*>(&sample_kernel_row<1>)
                              : reinterpret_cast<const void*>(&sample_kernel_row<0>);
  SampleParams copy = p;
  void* args[] = {&copy};
  return cudaLaunchKernel(fn, dim3(p.R), dim3(kThreads), args, sizeof(Smem), stream);
}

}  // namespace sv
