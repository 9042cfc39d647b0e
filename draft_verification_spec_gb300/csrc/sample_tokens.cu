// Sampling with temperature, top-k, top-p and min-p from given uniforms.
//
// A row's tokens are taken in the order (logit descending, index ascending).  With weights
// w = 2^((z - max) c), c = log2(e) / T, each filter keeps a prefix of that order:
//   top-k   the first k;
//   top-p   of those, the shortest prefix whose weight reaches top_p x the weight of the k;
//   min-p   the tokens with w >= min_p (the largest w is 1);
// the kept ones are the first n = min of the three (at least one), and the drawn token is the first
// whose inclusive prefix weight is strictly above u x the weight of the n.  Every question is "which
// element of the order does a count or a weight reach".
//
// One CTA per row, or, where rows are few, a cluster of CTAs (`Cl`) with a share of the row each: histograms
// are added up over the cluster, and every CTA goes on with the same sums.  A histogram over the 16 top
// bits of the logits (those of magnitude 2^-32 to 2^8, in descending order, and zero: 10,242 bins)
// answers it: the non-empty bins, a few hundred to a few thousand, become a list whose counts and
// weights are summed once over the block, and a question is a search in those sums.  A bf16 bin is one
// value, so its weight is count x weight and the row needs neither its maximum first nor an exponential
// per token.  An fp32 bin also sums its tokens' weights, and the element is then found among the bin's
// own by the digits of its low 16 bits.
// Rows with logits outside the bins' range (nothing sensible has them) go the general way: a descent
// over all digits of the ordered keys, 11 bits at a time.
// Equal logits are told apart by their index in a last ordered pass, which also writes the filtered row.
//
// Bound: the latency of the phases (histogram, list, searches, index, filtered row) at two rows an SM.  1088
// rows of 128000 bf16 with the filtered rows (557 MB) take 222 us, 37 % of the measured copy; a quarter of that is
// the histogram, whose shared-memory atomics are not what limits it (77 us for the rows with them, 61 without).
#include <atomic>
#include <cuda_bf16.h>

#include "sample_weight.cuh"
#include "spec_async.cuh"
#include "step_internal.h"

namespace sv {

namespace {

constexpr int kDigitBits = 11, kBins = 1 << kDigitBits;   // the general descent
constexpr int kMagLow = (127 - 32) * 128, kMags = 40 * 128;   // magnitudes of the histogram, in 7-bit mantissa steps
constexpr int kHist = 2 * kMags + 2;                      // positive, zero, negative, below -2^8
constexpr int kZeroBin = kMags, kLowBin = kHist - 1;
constexpr int kOutside = kHist + 1;                       // the histogram's word for logits without a bin (word kHist stays zero)

constexpr int kGather = 8192;                             // fp32: tokens of one bin that are looked through in shared memory

template <int DTYPE>
struct Geo;
template <>
struct Geo<1> {   // bf16: counts only
  using Raw = uint16_t;
  // 512 threads: 222 us for 1088 rows of 128000 with the filtered rows; 256: 260, 384: 243, 1024: 256 us
  static constexpr int kThreads = 512, kVec = 8, kPer = 21;   // bins per thread: odd, so a warp's reads fall on distinct banks
  static constexpr int kHistWords = kThreads * kPer;
  static constexpr int kDigitWords = 0;                   // the general descent reuses the histogram
};
template <>
struct Geo<0> {   // fp32: counts and weights
  using Raw = uint32_t;
  static constexpr int kThreads = 1024, kVec = 4, kPer = 11;
  static constexpr int kHistWords = 3 * kThreads * kPer;
  static constexpr int kDigitWords = 3 * kBins + kGather;
};
static_assert(Geo<1>::kThreads * Geo<1>::kPer > kHist + 1 && Geo<0>::kThreads * Geo<0>::kPer > kHist + 1, "every bin has a thread");
static_assert(Geo<1>::kHistWords >= 3 * kBins, "the general descent fits the histogram");

template <int DTYPE>
constexpr int smem_bytes() {
  return 4 * (Geo<DTYPE>::kHistWords + Geo<DTYPE>::kDigitWords) + 2 * ((kHist + 7) / 8 * 8);
}

template <int DTYPE>
__device__ __forceinline__ float value_of(typename Geo<DTYPE>::Raw b) {
  return __uint_as_float(DTYPE == 1 ? static_cast<uint32_t>(b) << 16 : static_cast<uint32_t>(b));
}
// Ordered key, right-aligned (16 or 32 bits); NaN counts as -inf, which is never drawn.
template <int DTYPE>
__device__ __forceinline__ uint32_t sample_key(float z) {
  const uint32_t k = ord_key(z != z ? ninf() : z);
  return DTYPE == 1 ? k >> 16 : k;
}
template <int DTYPE>
__device__ __forceinline__ float key_value(uint32_t k) {
  if (DTYPE == 1) k = k << 16 | (k & 0x8000u ? 0u : 0xffffu);
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// Bins are numbered in the order's direction; in the histogram, where the fast path has three
// instructions for a logit's place, the positive magnitudes come first, then the negative ones, zero
// and those below -2^8.
__device__ __forceinline__ int place_of(int bin) {
  return bin < kZeroBin ? kZeroBin - 1 - bin : bin == kZeroBin ? 2 * kMags : bin == kLowBin ? kLowBin : bin - 1;
}
__device__ __forceinline__ unsigned place_in_range(uint32_t top) {   // top: 16 bits, magnitude in the bins' range
  return top + (top >> 15) * static_cast<unsigned>(kMags - 0x8000) - kMagLow;
}
// Of the other logits: zero, those below -2^8; -1 for -inf and NaN (never drawn), -2 for what has no bin.
template <int DTYPE>
__device__ __forceinline__ int place_other(typename Geo<DTYPE>::Raw b) {
  const uint32_t bits = DTYPE == 1 ? static_cast<uint32_t>(b) << 16 : static_cast<uint32_t>(b), mag = bits & 0x7fffffffu;
  if (mag == 0u) return 2 * kMags;
  if (mag > 0x7f800000u || bits == 0xff800000u) return -1;
  return static_cast<int>(mag >> 16) >= kMagLow + kMags && (bits >> 31) ? kLowBin : -2;
}
// A bin's value with the lowest magnitude (bf16: its value); its key's 16 top bits.
__device__ __forceinline__ float bin_value(int bin) {
  if (bin == kZeroBin) return 0.f;
  const uint32_t top = bin < kZeroBin ? kMagLow + (kZeroBin - 1 - bin) : 0x8000u | (kMagLow + (bin - kZeroBin - 1));
  return __uint_as_float(top << 16);
}
__device__ __forceinline__ uint32_t bin_key16(int bin) {
  if (bin == kZeroBin) return 0x8000u;
  return bin < kZeroBin ? 0x8000u | (kMagLow + (kZeroBin - 1 - bin)) : 0x7fffu & ~static_cast<uint32_t>(kMagLow + (bin - kZeroBin - 1));
}

// A row in units of one 16-byte piece: unit 0 is what lies before the first 16-byte boundary (possibly
// nothing), the last one what lies behind the last.
template <int DTYPE>
struct Row {
  using Raw = typename Geo<DTYPE>::Raw;
  static constexpr int VEC = Geo<DTYPE>::kVec;
  const Raw* p;
  int V, head, full, units;   // units 1 .. full are whole pieces
  int u0, u1;                 // this CTA's units
  __device__ __forceinline__ Row(const void* base, int v, int rank, int ctas) : p(static_cast<const Raw*>(base)), V(v) {
    const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(base) & 15u) / static_cast<int>(sizeof(Raw));
    head = min(V, mis ? VEC - mis : 0);
    full = (V - head) / VEC;
    units = full + 2;
    u0 = units * rank / ctas;
    u1 = units * (rank + 1) / ctas;
  }
  __device__ __forceinline__ bool whole(int u) const { return u > 0 && u <= full; }
  __device__ __forceinline__ int first(int u) const { return u == 0 ? 0 : head + (u - 1) * VEC; }
  __device__ __forceinline__ int count(int u) const { return u == 0 ? head : min(VEC, V - first(u)); }
  // the first or the last unit's values; places beyond its count hold -inf
  __device__ __noinline__ uint4 edge(int u) const {
    Raw x[VEC];
    const int i0 = first(u), n = count(u);
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = e < n ? __ldg(p + i0 + e) : static_cast<Raw>(DTYPE == 1 ? 0xff80u : 0xff800000u);
    uint4 v;
    memcpy(&v, x, 16);
    return v;
  }
  // a whole piece near unit u (for the edges any one; zeros if there is none): a load without a branch
  __device__ __forceinline__ uint4 near(int u) const {
    return full > 0 ? __ldg(reinterpret_cast<const uint4*>(p + head) + min(max(u - 1, 0), full - 1)) : make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ uint4 load(int u) const { return whole(u) ? near(u) : edge(u); }
  static __device__ __forceinline__ Raw value(const uint4& v, int e) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    return DTYPE == 1 ? static_cast<Raw>(w[e / 2] >> (16 * (e & 1))) : static_cast<Raw>(w[e & 3]);
  }
};

// f(unit, piece) for the units [begin, end) in steps of `stride`, BATCH loads in flight at a time.
template <int DTYPE, int BATCH, typename F>
__device__ __forceinline__ void walk(const Row<DTYPE>& row, int begin, int end, int stride, F f) {
  for (int u = begin; u < end; u += BATCH * stride) {
    uint4 x[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) x[i] = row.near(u + i * stride);
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int at = u + i * stride;
      if (at >= end) break;
      if (!row.whole(at)) x[i] = row.edge(at);
      f(at, x[i]);
    }
  }
}

// How many of a piece's values equal v; which are greater (masks of the values' width).
template <int DTYPE>
struct Compare;
template <>
struct Compare<1> {
  __nv_bfloat162 v;
  __device__ __forceinline__ explicit Compare(float x) : v(__float2bfloat162_rn(x)) {}
  __device__ __forceinline__ unsigned eq(uint32_t w) const { return __heq2_mask(*reinterpret_cast<__nv_bfloat162*>(&w), v); }
  __device__ __forceinline__ unsigned gt(uint32_t w) const { return __hgt2_mask(*reinterpret_cast<__nv_bfloat162*>(&w), v); }
  static constexpr unsigned kOnes = 0x00010001u, kDropWord = 0xff80ff80u;
  static __device__ __forceinline__ unsigned total(unsigned packed) { return (packed & 0xffffu) + (packed >> 16); }
};
template <>
struct Compare<0> {
  float v;
  __device__ __forceinline__ explicit Compare(float x) : v(x) {}
  __device__ __forceinline__ unsigned eq(uint32_t w) const { return __uint_as_float(w) == v ? 0xffffffffu : 0u; }
  __device__ __forceinline__ unsigned gt(uint32_t w) const { return __uint_as_float(w) > v ? 0xffffffffu : 0u; }
  static constexpr unsigned kOnes = 1u, kDropWord = 0xff800000u;
  static __device__ __forceinline__ unsigned total(unsigned packed) { return packed; }
};

struct Prefix {
  unsigned cnt;            // tokens before the group in the order
  unsigned long long mass;
  uint32_t key;            // the group's key (or its place in the bins' list)
};

template <int NT, bool Cl>
struct Shared {
  unsigned long long tab[64];
  unsigned long long wmass[32];
  unsigned wcnt[32], wcnt2[32];
  Prefix found;
  float c_hi, c_lo;                  // the scale of the weights
  unsigned long long least, target;  // min-p's weight; the weight that is looked for
  float prob;
  unsigned group_in;                 // how many of a group's tokens reach the target
  int token;
  unsigned gathered;
  // what the CTAs of a cluster tell one another, in two places in turn
  int rank, ctas, turn;
  struct {
    unsigned a, b;
    unsigned long long m;
    float top;
  } said[2];
};

template <typename T>
__device__ __forceinline__ const T* of_peer(const T* p, int rank) {
  const T* q;
  asm volatile("mapa.u64 %0, %1, %2;" : "=l"(q) : "l"(p), "r"(rank));
  return q;
}

// Sums over the cluster (`lower`: over the CTAs before this one) and its largest value, with one cluster
// barrier: what was said last but one has been read by everybody who passed the last one.
template <int NT, bool Cl>
__device__ __noinline__ float cluster_sum(unsigned& a, unsigned& b, unsigned long long& m, float top, bool lower, Shared<NT, Cl>& s) {
  const int t = s.turn;
  if (threadIdx.x == 0) s.said[t].a = a, s.said[t].b = b, s.said[t].m = m, s.said[t].top = top;
  cluster_sync();
  a = b = 0u;
  m = 0ull;
  for (int r = 0; r < s.ctas; ++r) {
    const auto* o = of_peer(&s.said[t], r);
    top = fmaxf(top, o->top);
    if (lower && r >= s.rank) continue;
    a += o->a;
    b += o->b;
    m += o->m;
  }
  __syncthreads();
  if (threadIdx.x == 0) s.turn = t ^ 1;
  __syncthreads();
  return top;
}

// Adds up the cluster's copies of an array of 4 n counts and, behind it (weights), of the low and high words
// of 4 n 64-bit sums.  Every CTA sums a share, then fetches the others'.
template <int NT, bool Cl>
__device__ __noinline__ void cluster_merge(unsigned* words, int n, bool weights, Shared<NT, Cl>& s) {
  uint4* c = reinterpret_cast<uint4*>(words);
  const int me = s.rank, i0 = n * me / s.ctas, i1 = n * (me + 1) / s.ctas;
  cluster_sync();
  for (int i = i0 + threadIdx.x; i < i1; i += NT) {
    uint4 x = c[i], lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
    if (weights) lo = c[n + i], hi = c[2 * n + i];
    for (int k = 1; k < s.ctas; ++k) {
      const uint4* o = of_peer(c, (me + k) % s.ctas);
      const uint4 y = o[i];
      x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
      if (weights) {
        const uint4 l = o[n + i], h = o[2 * n + i];
        lo.x += l.x, lo.y += l.y, lo.z += l.z, lo.w += l.w;
        hi.x += h.x + (lo.x < l.x), hi.y += h.y + (lo.y < l.y), hi.z += h.z + (lo.z < l.z), hi.w += h.w + (lo.w < l.w);
      }
    }
    c[i] = x;
    if (weights) c[n + i] = lo, c[2 * n + i] = hi;
  }
  cluster_sync();
  for (int k = 1; k < s.ctas; ++k) {
    const int r = (me + k) % s.ctas, j0 = n * r / s.ctas, j1 = n * (r + 1) / s.ctas;
    const uint4* o = of_peer(c, r);
    for (int i = j0 + threadIdx.x; i < j1; i += NT) {
      c[i] = o[i];
      if (weights) c[n + i] = o[n + i], c[2 * n + i] = o[2 * n + i];
    }
  }
  cluster_sync();   // nobody changes its words before all have fetched them
}

// Block-wide exclusive prefix of (count, weight); the totals too.
template <int NT, bool Cl>
__device__ __forceinline__ void block_scan(unsigned& c, unsigned long long& m, unsigned* c_all, unsigned long long* m_all,
                                           Shared<NT, Cl>& s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned ic = c;
  unsigned long long im = m;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned tc = __shfl_up_sync(0xffffffffu, ic, o);
    const unsigned long long tm = __shfl_up_sync(0xffffffffu, im, o);
    if (lane >= o) ic += tc, im += tm;
  }
  if (lane == 31) s.wcnt[warp] = ic, s.wmass[warp] = im;
  __syncthreads();
  unsigned wc = lane < NT / 32 ? s.wcnt[lane] : 0u;
  unsigned long long wm = lane < NT / 32 ? s.wmass[lane] : 0ull;
#pragma unroll
  for (int o = 1; o < NT / 32; o <<= 1) {
    const unsigned tc = __shfl_up_sync(0xffffffffu, wc, o);
    const unsigned long long tm = __shfl_up_sync(0xffffffffu, wm, o);
    if (lane >= o) wc += tc, wm += tm;
  }
  const unsigned bc = __shfl_sync(0xffffffffu, wc, warp > 0 ? warp - 1 : 0);
  const unsigned long long bm = __shfl_sync(0xffffffffu, wm, warp > 0 ? warp - 1 : 0);
  *c_all = __shfl_sync(0xffffffffu, wc, NT / 32 - 1);
  *m_all = __shfl_sync(0xffffffffu, wm, NT / 32 - 1);
  c = (warp > 0 ? bc : 0u) + ic - c;
  m = (warp > 0 ? bm : 0ull) + im - m;
  __syncthreads();
}

// Adds a weight to a pair of words; the carry goes up.
__device__ __forceinline__ void add_weight(unsigned* lo, unsigned* hi, unsigned long long w) {
  const unsigned l = static_cast<unsigned>(w);
  const unsigned old = atomicAdd(lo, l);
  const unsigned up = static_cast<unsigned>(w >> 32) + (old + l < old ? 1u : 0u);
  if (up) atomicAdd(hi, up);
}

// Block-wide: the group of equal keys in which the order's count or weight reaches `target` (1 <= target
// <= the row's), among the tokens whose key begins with at.key, `bits` bits being open.  With `gathered`
// >= 0 those tokens' keys are in `keys`, else the row is read, once per 11 bits.
template <int DTYPE, bool Cl>
__device__ __noinline__ Prefix descend(const Row<DTYPE>& row, const WeightScale& ws, bool by_count, unsigned long long target,
                                       Prefix at, int bits, unsigned* digits, const uint32_t* keys, int gathered,
                                       Shared<Geo<DTYPE>::kThreads, Cl>& s) {
  constexpr int NT = Geo<DTYPE>::kThreads, PER = kBins / NT, VEC = Geo<DTYPE>::kVec;
  const int tid = threadIdx.x;
  unsigned *cnt = digits, *lo = digits + kBins, *hi = digits + 2 * kBins;
  while (bits > 0) {
    const int digit = bits < kDigitBits ? bits : kDigitBits;
    bits -= digit;
    for (int i = tid; i < 3 * kBins; i += NT) digits[i] = 0u;
    __syncthreads();
    auto take = [&](uint32_t key, float z) {
      if ((static_cast<unsigned long long>(key) >> (bits + digit)) != at.key || !(z > ninf())) return;
      const unsigned d = (key >> bits) & ((1u << digit) - 1u);
      atomicAdd(&cnt[d], 1u);
      add_weight(&lo[d], &hi[d], weight_of(z, ws, s.tab));
    };
    if (gathered >= 0) {
      for (int i = tid; i < gathered; i += NT) take(keys[i], key_value<DTYPE>(keys[i]));
    } else {
      walk<DTYPE, 2>(row, row.u0 + tid, row.u1, NT, [&](int, const uint4& piece) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float z = value_of<DTYPE>(Row<DTYPE>::value(piece, e));
          take(sample_key<DTYPE>(z), z);
        }
      });
    }
    __syncthreads();
    if (Cl && gathered < 0) cluster_merge<NT, Cl>(digits, kBins / 4, true, s);
    // thread t holds PER bins from the top
    unsigned c[PER], bc = 0, all_c;
    unsigned long long m[PER], bm = 0, all_m;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int bin = kBins - 1 - (PER * tid + e);
      c[e] = cnt[bin];
      m[e] = (static_cast<unsigned long long>(hi[bin]) << 32) + lo[bin];
      bc += c[e];
      bm += m[e];
    }
    block_scan<NT, Cl>(bc, bm, &all_c, &all_m, s);
    bc += at.cnt;
    bm += at.mass;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const bool before = by_count ? bc < target : bm < target;
      const bool reached = by_count ? bc + c[e] >= target : bm + m[e] >= target;
      if (before && reached) s.found = {bc, bm, static_cast<uint32_t>((at.key << digit) | (kBins - 1 - (PER * tid + e)))};
      bc += c[e];
      bm += m[e];
    }
    __syncthreads();
    at = s.found;
    __syncthreads();
  }
  return at;
}

// fp32, block-wide: the same among the tokens of one bin (16 open bits), whose keys are gathered first.
template <int DTYPE, bool Cl>
__device__ __noinline__ Prefix descend_bin(const Row<DTYPE>& row, const WeightScale& ws, bool by_count,
                                           unsigned long long target, Prefix at, unsigned tokens, unsigned* digits,
                                           Shared<Geo<DTYPE>::kThreads, Cl>& s) {
  constexpr int NT = Geo<DTYPE>::kThreads, VEC = Geo<DTYPE>::kVec;
  uint32_t* keys = digits + 3 * kBins;
  if (tokens > kGather) return descend<DTYPE, Cl>(row, ws, by_count, target, at, 16, digits, nullptr, -1, s);
  if (threadIdx.x == 0) s.gathered = 0u;
  __syncthreads();
  // the bin's logits by their bits: 16 top bits, or zero of either sign
  const bool zero = at.key == 0x8000u;
  const uint32_t want = zero ? 0u : (at.key & 0x8000u ? at.key & 0x7fffu : 0xffffu & ~at.key);
  const int shift = zero ? 0 : 16;
  walk<DTYPE, 4>(row, row.u0 + threadIdx.x, row.u1, NT, [&](int, const uint4& piece) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const uint32_t x = Row<DTYPE>::value(piece, e);
      if ((zero ? x & 0x7fffffffu : x) >> shift == want) keys[atomicAdd(&s.gathered, 1u)] = sample_key<DTYPE>(value_of<DTYPE>(x));
    }
  });
  __syncthreads();
  if (Cl) {   // the others' keys behind one's own
    cluster_sync();
    unsigned have = s.gathered;
    for (int k = 1; k < s.ctas; ++k) {
      const int r = (s.rank + k) % s.ctas;
      const unsigned n = *of_peer(&s.gathered, r);
      const uint32_t* o = of_peer(keys, r);
      for (unsigned i = threadIdx.x; i < n; i += NT) keys[have + i] = o[i];
      have += n;
    }
    cluster_sync();   // nobody gathers again before all have copied
  }
  return descend<DTYPE, Cl>(row, ws, by_count, target, at, 16, digits, keys, static_cast<int>(tokens), s);
}

// Block-wide largest logit (NaN left out).
template <int DTYPE, bool Cl>
__device__ __noinline__ float row_max(const Row<DTYPE>& row, Shared<Geo<DTYPE>::kThreads, Cl>& s) {
  constexpr int NT = Geo<DTYPE>::kThreads, VEC = Geo<DTYPE>::kVec;
  float top = ninf();
  walk<DTYPE, 4>(row, row.u0 + threadIdx.x, row.u1, NT, [&](int, const uint4& piece) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) top = fmaxf(top, value_of<DTYPE>(Row<DTYPE>::value(piece, e)));
  });
  top = warp_max(top);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s.wcnt2[threadIdx.x >> 5] = __float_as_uint(top);
  __syncthreads();
  for (int w = 0; w < NT / 32; ++w) top = fmaxf(top, __uint_as_float(s.wcnt2[w]));
  __syncthreads();
  if (Cl) {
    unsigned a = 0, b = 0;
    unsigned long long m = 0;
    top = cluster_sum<NT, Cl>(a, b, m, top, false, s);
  }
  return top;
}

struct Totals {
  unsigned n_all, n_min;               // tokens above -inf, those of at least min-p's weight
  unsigned long long m_all, m_min;     // their weights
};

// The general way's totals.
template <int DTYPE, bool Cl>
__device__ __noinline__ Totals row_totals(const Row<DTYPE>& row, const WeightScale& ws, unsigned long long least,
                                          Shared<Geo<DTYPE>::kThreads, Cl>& s) {
  constexpr int NT = Geo<DTYPE>::kThreads, VEC = Geo<DTYPE>::kVec;
  Totals t = {0u, 0u, 0ull, 0ull};
  walk<DTYPE, 1>(row, row.u0 + threadIdx.x, row.u1, NT, [&](int, const uint4& piece) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float z = value_of<DTYPE>(Row<DTYPE>::value(piece, e));
      if (!(z > ninf())) continue;
      const unsigned long long w = weight_of(z, ws, s.tab);
      ++t.n_all;
      t.m_all += w;
      if (w >= least) ++t.n_min, t.m_min += w;
    }
  });
  unsigned c = t.n_all;
  unsigned long long m = t.m_all;
  block_scan<NT, Cl>(c, m, &t.n_all, &t.m_all, s);
  if (Cl) {
    unsigned none = 0;
    cluster_sum<NT, Cl>(t.n_all, none, t.m_all, 0.f, false, s);
  }
  return t;
}

// A thread's share [i0, i1) of the list of non-empty bins, and what lies before it.
template <int DTYPE>
struct Bins {
  static constexpr int SPAN = Geo<DTYPE>::kThreads * Geo<DTYPE>::kPer;
  const unsigned* hist;
  const uint16_t* list;
  unsigned* digits;
  int i0, i1;
  unsigned cnt;
  unsigned long long mass;
  bool general;
  // weight of one token (bf16) or of the whole bin (fp32)
  __device__ __forceinline__ unsigned long long weight(int b, const WeightScale& ws, const unsigned long long* tab) const {
    if (DTYPE == 0) return (static_cast<unsigned long long>(hist[2 * SPAN + place_of(b)]) << 32) + hist[SPAN + place_of(b)];
    return b == kLowBin ? 0ull : weight_of(bin_value(b), ws, tab);
  }
};

// A group of equal logits, what lies before it in the order, a token's weight.
struct Group {
  float z;
  unsigned cnt;
  unsigned long long mass, w;
};

// Block-wide: the group in which the order's count or weight reaches the target.
template <int DTYPE, bool Cl>
__device__ __noinline__ Group reach(const Row<DTYPE>& row, const WeightScale& ws, Bins<DTYPE>& bins, bool by_count,
                                    unsigned long long target, Shared<Geo<DTYPE>::kThreads, Cl>& s) {
  constexpr int kBitsAll = DTYPE == 1 ? 16 : 32;
  Prefix g = {0u, 0ull, 0u};
  if (bins.general) {
    g = descend<DTYPE, Cl>(row, ws, by_count, target, g, kBitsAll, bins.digits, nullptr, -1, s);
  } else {
    unsigned c = bins.cnt;
    unsigned long long m = bins.mass;
    for (int i = bins.i0; i < bins.i1; ++i) {
      if (by_count ? c >= target : m >= target) break;
      const int b = bins.list[i];
      const unsigned bc = bins.hist[place_of(b)];
      const unsigned long long w = bins.weight(b, ws, s.tab), bm = DTYPE == 1 ? bc * w : w;
      if (by_count ? c + bc >= target : m + bm >= target) s.found = {c, m, static_cast<uint32_t>(b)};
      c += bc;
      m += bm;
    }
    __syncthreads();
    g = s.found;
    __syncthreads();
    if (DTYPE == 1 && g.key != kLowBin) {
      const float z = bin_value(g.key);
      return {z, g.cnt, g.mass, weight_of(z, ws, s.tab)};
    }
    if (g.key == kLowBin) {
      // among the logits below -2^8 (a count went there): their weights are zero, all digits are open.
      // In bf16 the descent's histogram takes the list's place: later questions go the general way.
      const Prefix low = {0u, 0ull, 0u};
      g = descend<DTYPE, Cl>(row, ws, true, target, low, kBitsAll, bins.digits, nullptr, -1, s);
      if (DTYPE == 1) bins.general = true;
    } else {
      const unsigned tokens = bins.hist[place_of(g.key)];
      g.key = bin_key16(g.key);
      g = descend_bin<DTYPE, Cl>(row, ws, by_count, target, g, tokens, bins.digits, s);
    }
  }
  const float z = key_value<DTYPE>(g.key);
  return {z, g.cnt, g.mass, weight_of(z, ws, s.tab)};
}

template <int DTYPE, bool Cl>
__global__ void __launch_bounds__(Geo<DTYPE>::kThreads, DTYPE == 1 ? 2 : 1) sample_kernel_row(const SampleParams p) {
  using G = Geo<DTYPE>;
  using Raw = typename G::Raw;
  constexpr int NT = G::kThreads, VEC = G::kVec, PER = G::kPer, NW = NT / 32, SPAN = NT * PER;
  extern __shared__ __align__(16) unsigned dyn[];
  unsigned* hist = dyn;                                           // [SPAN] counts (fp32: then weights, low and high words)
  unsigned* digits = DTYPE == 1 ? dyn : dyn + G::kHistWords;      // the general descent's
  uint16_t* list = reinterpret_cast<uint16_t*>(dyn + G::kHistWords + G::kDigitWords);   // non-empty bins
  __shared__ Shared<NT, Cl> s;
  const int ctas = Cl ? static_cast<int>(cluster_ncta()) : 1, cta = Cl ? static_cast<int>(cluster_rank()) : 0;
  const int r = blockIdx.x / ctas, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Row<DTYPE> row(static_cast<const Raw*>(p.logits) + static_cast<long long>(r) * p.stride, p.V, cta, ctas);

  float T = p.temperature ? p.temperature[r] : p.temperature0;
  int k = p.top_k ? p.top_k[r] : p.top_k0;
  const float top_p = p.top_p ? p.top_p[r] : p.top_p0, min_p = p.min_p ? p.min_p[r] : p.min_p0;
  const float uniform = p.uniforms[r];
  if (!(T > 0.f)) {   // greedy: the first of the order
    T = 1.f;
    k = 1;
  }
  if (tid < 64) s.tab[tid] = kExp2Table[tid];
  if (tid == 0) {   // 64-bit floating point is slow here: one thread does what there is of it
    s.rank = cta;
    s.ctas = ctas;
    s.turn = 0;
    s.token = -1;
    const WeightScale w = weight_scale(0.f, T);
    s.c_hi = w.c_hi;
    s.c_lo = w.c_lo;
    s.least = min_p > 0.f ? static_cast<unsigned long long>(ceil(static_cast<double>(min_p) * kWeightOne)) : 0ull;
  }
  __syncthreads();
  const bool need_max = DTYPE == 0 || k == 1;
  const bool filter = p.filtered != nullptr;

  // the largest logit, where it is needed before the weights
  float zmax = need_max ? row_max<DTYPE, Cl>(row, s) : ninf();

  // what the last pass needs: the drawn value and its rank among its equals, the cut's value and how
  // many of its equals are kept
  unsigned n = 0, rank = 0, cut_eq = 0;
  float z_draw = 0.f, z_cut = 0.f, prob = 0.f;
  bool any = true, whole_ties = true;   // whole_ties: every token equal to the cut's is kept
  if (k == 1) {
    any = zmax > ninf();
    n = any ? 1u : 0u;
    z_draw = z_cut = zmax;
    cut_eq = 1;
    whole_ties = false;
    prob = any ? 1.f : 0.f;
  } else {
    // histogram
    for (int i = tid; i < G::kHistWords / 4; i += NT) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    WeightScale ws = {zmax, s.c_hi, s.c_lo};
    const unsigned long long least = s.least;
    unsigned n_min = 0, n_all;
    unsigned long long m_min = 0, m_all;
    bool out_of_range = false;
    const bool count_min = min_p > 0.f;
    auto count = [&](Raw x, unsigned at) {
      atomicAdd(&hist[at], 1u);
      if (DTYPE == 0) {
        const unsigned long long w = weight_of(value_of<DTYPE>(x), ws, s.tab);
        if (w) add_weight(&hist[SPAN + at], &hist[2 * SPAN + at], w);
        if (count_min && w >= least) ++n_min, m_min += w;
      }
    };
    walk<DTYPE, 4>(row, row.u0 + tid, row.u1, NT, [&](int, const uint4& piece) {
      bool fast = true;   // all of the piece in the bins' range
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const uint32_t x = Row<DTYPE>::value(piece, e), top = DTYPE == 1 ? x : x >> 16;
        fast = fast && (top & 0x7fffu) - kMagLow < static_cast<unsigned>(kMags);
      }
      if (fast) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const Raw x = Row<DTYPE>::value(piece, e);
          count(x, place_in_range(DTYPE == 1 ? x : static_cast<uint32_t>(x) >> 16));
        }
      } else {
#pragma unroll 1
        for (int e = 0; e < VEC; ++e) {
          const uint32_t word = DTYPE == 1 ? (e < 4 ? (e < 2 ? piece.x : piece.y) : (e < 6 ? piece.z : piece.w)) >> (16 * (e & 1))
                                           : (e < 2 ? (e < 1 ? piece.x : piece.y) : (e < 3 ? piece.z : piece.w));
          const Raw x = static_cast<Raw>(word);
          const uint32_t top = DTYPE == 1 ? x : static_cast<uint32_t>(x) >> 16;
          const int at = (top & 0x7fffu) - kMagLow < static_cast<unsigned>(kMags) ? static_cast<int>(place_in_range(top)) : place_other<DTYPE>(x);
          if (at >= 0) count(x, at);
          out_of_range |= at == -2;
        }
      }
    });
    if (out_of_range) atomicAdd(&hist[kOutside], 1u);
    __syncthreads();
    if (Cl) cluster_merge<NT, Cl>(hist, SPAN / 4, DTYPE == 0, s);
    // the non-empty bins, in order
    static_assert(PER <= 32, "a bit per bin");
    unsigned filled = 0, listed;   // this thread's bins that are not empty
    unsigned long long none = 0, none_all;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int bin = min(tid * PER + e, kHist);   // the word behind the bins is zero
      filled |= (hist[bin == kHist ? kHist : place_of(bin)] != 0u ? 1u : 0u) << e;
    }
    unsigned at = __popc(filled);
    block_scan<NT, Cl>(at, none, &listed, &none_all, s);
    for (unsigned left = filled; left; left &= left - 1) list[at++] = static_cast<uint16_t>(tid * PER + __ffs(left) - 1);
    __syncthreads();
    if (DTYPE == 1 && listed > 0) {
      zmax = bin_value(list[0]);
      ws.zmax = zmax;
    }
    Bins<DTYPE> bins;
    const int share = (listed + NT - 1) / NT;
    bins.hist = hist;
    bins.list = list;
    bins.digits = digits;
    bins.i0 = min(static_cast<int>(listed), tid * share);
    bins.i1 = min(static_cast<int>(listed), bins.i0 + share);
    bins.cnt = 0u;
    bins.mass = 0ull;
    // below -2^8 the weights have to be zero (one unknown weight would be wrong)
    bins.general = hist[kOutside] || (listed > 0 && (list[0] == kLowBin || (hist[kLowBin] && weight_of(-256.f, ws, s.tab) != 0ull)));
    if (!bins.general) {
      for (int i = bins.i0; i < bins.i1; ++i) {
        const int b = list[i];
        const unsigned c = hist[place_of(b)];
        const unsigned long long w = bins.weight(b, ws, s.tab);
        bins.cnt += c;
        bins.mass += DTYPE == 1 ? c * w : w;
        if (DTYPE == 1 && w >= least) n_min += c, m_min += c * w;
      }
      block_scan<NT, Cl>(bins.cnt, bins.mass, &n_all, &m_all, s);
    } else {
      ws.zmax = row_max<DTYPE, Cl>(row, s);
      const Totals t = row_totals<DTYPE, Cl>(row, ws, least, s);
      n_all = t.n_all;
      m_all = t.m_all;
      n_min = t.n_min;
      m_min = t.m_min;
    }
    if (min_p > 0.f) {
      unsigned c = n_min, none = 0;
      unsigned long long m = m_min;
      block_scan<NT, Cl>(c, m, &n_min, &m_min, s);
      if (Cl && (DTYPE == 0 || bins.general)) cluster_sum<NT, Cl>(n_min, none, m_min, 0.f, false, s);   // else: counted from the merged bins
    }
    any = n_all > 0;
    if (any) {
      n = n_all;
      unsigned long long mass = m_all;
      Group cut = {0.f, 0u, 0ull, 0ull};
      bool cut_known = false;
      if (k > 0 && static_cast<unsigned>(k) < n) {
        cut = reach<DTYPE, Cl>(row, ws, bins, true, k, s);
        cut_known = true;
        n = k;
        mass = cut.mass + (k - cut.cnt) * cut.w;
      }
      if (top_p < 1.f) {
        if (tid == 0) {
          const double goal = ceil(fmax(static_cast<double>(top_p), 0.0) * static_cast<double>(mass));
          const unsigned long long t = goal < 1.0 ? 1ull : static_cast<unsigned long long>(goal);
          s.target = t > mass ? mass : t;
        }
        __syncthreads();
        const unsigned long long target = s.target;
        const Group g = reach<DTYPE, Cl>(row, ws, bins, false, target, s);
        if (tid == 0) s.group_in = static_cast<unsigned>((target - g.mass + g.w - 1) / g.w);
        __syncthreads();
        const unsigned in = s.group_in;
        if (g.cnt + in < n) {
          n = g.cnt + in;
          mass = g.mass + in * g.w;
          cut = g;
          cut_known = true;
        }
      }
      if (min_p > 0.f && n_min < n) {
        n = n_min > 0 ? n_min : 1;
        mass = n_min > 0 ? m_min : kWeightOne;
        cut_known = false;
      }
      // the draw
      if (tid == 0) {
        const double td = uniform > 0.f ? floor(static_cast<double>(uniform) * static_cast<double>(mass)) : 0.0;
        const unsigned long long t = td >= static_cast<double>(mass) ? mass - 1 : static_cast<unsigned long long>(td);
        s.target = (t >= mass ? mass - 1 : t) + 1;
      }
      __syncthreads();
      const unsigned long long target = s.target;
      const Group g = reach<DTYPE, Cl>(row, ws, bins, false, target, s);
      if (tid == 0) {
        s.group_in = static_cast<unsigned>((target - g.mass + g.w - 1) / g.w);
        s.prob = static_cast<float>(static_cast<double>(g.w) / static_cast<double>(mass));
      }
      __syncthreads();
      z_draw = g.z;
      rank = s.group_in - 1;
      prob = s.prob;
      if (filter) {
        if (n == n_all) {
          z_cut = ninf();   // everything above -inf stays
        } else {
          if (!cut_known) cut = reach<DTYPE, Cl>(row, ws, bins, true, n, s);
          z_cut = cut.z;
          cut_eq = n - cut.cnt;
          whole_ties = false;
        }
      }
    }
  }

  // ordered passes: warp w takes a contiguous share of the units, so that equal logits can be counted in
  // index order.  First the equal ones per warp, then the drawn token, then the filtered row.
  const int per_warp = (row.u1 - row.u0 + NW - 1) / NW;
  const int u0 = min(row.u1, row.u0 + warp * per_warp), u1 = min(row.u1, u0 + per_warp);
  if (any) {
    unsigned eq = 0, eq_cut = 0;
    const Compare<DTYPE> drawn(z_draw), cutoff(z_cut);
    const bool ordered = filter && !whole_ties;
    walk<DTYPE, 4>(row, u0 + lane, u1, 32, [&](int, const uint4& piece) {
      const uint32_t w[4] = {piece.x, piece.y, piece.z, piece.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        eq += drawn.eq(w[e]) & Compare<DTYPE>::kOnes;
        if (ordered) eq_cut += cutoff.eq(w[e]) & Compare<DTYPE>::kOnes;
      }
    });
    eq = Compare<DTYPE>::total(eq);
    eq_cut = Compare<DTYPE>::total(eq_cut);
    eq = __reduce_add_sync(0xffffffffu, eq);
    eq_cut = __reduce_add_sync(0xffffffffu, eq_cut);
    if (lane == 0) s.wcnt[warp] = eq, s.wcnt2[warp] = eq_cut;
    __syncthreads();
    unsigned before = 0, before_cut = 0;   // equal ones in the CTAs before this one, then in the warps too
    if (Cl) {
      unsigned long long none = 0;
      for (int w = 0; w < NW; ++w) before += s.wcnt[w], before_cut += s.wcnt2[w];
      cluster_sum<NT, Cl>(before, before_cut, none, 0.f, true, s);
    }
    int owner = rank >= before ? 0 : NW;
    for (int w = 0; w < NW; ++w) {
      if (w < warp) before_cut += s.wcnt2[w];
      if (owner == w && rank - before >= s.wcnt[w]) before += s.wcnt[w], ++owner;
    }
    __syncthreads();
    if (!Cl || owner < NW) {
      // the drawn token is in warp `owner`'s share: the whole block looks for it, each thread in
      // consecutive units
      const int o0 = min(row.u1, row.u0 + owner * per_warp), o1 = min(row.u1, o0 + per_warp);
      const int per = (o1 - o0 + NT - 1) / NT, a0 = min(o1, o0 + tid * per), a1 = min(o1, a0 + per);
      unsigned here = 0, all;
      unsigned long long none = 0, none_all;
      for (int u = a0; u < a1; ++u) {
        const uint4 piece = row.load(u);
#pragma unroll
        for (int e = 0; e < VEC; ++e) here += value_of<DTYPE>(Row<DTYPE>::value(piece, e)) == z_draw;
      }
      unsigned first = here;
      block_scan<NT, Cl>(first, none, &all, &none_all, s);
      const unsigned want = rank - before;
      if (want >= first && want < first + here) {
        unsigned skip = want - first;
        for (int u = a0; u < a1; ++u) {
          const uint4 piece = row.load(u);
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            if (value_of<DTYPE>(Row<DTYPE>::value(piece, e)) == z_draw && skip-- == 0) s.token = row.first(u) + e;
        }
      }
    }
    if (filter) {
      Raw* out = static_cast<Raw*>(p.filtered) + static_cast<long long>(r) * p.filtered_stride;
      // 16-byte stores where the output row lies as the input row does
      const bool vec = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(row.p)) & 15u) == 0;
      unsigned seen = before_cut;   // equal to the cut before this step of the warp
      constexpr int kAhead = 4;     // loads in flight
      for (int base = u0; base < u1; base += 32 * kAhead) {
        uint4 x[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) x[i] = row.near(base + i * 32 + lane);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int u = base + i * 32 + lane;
          const bool in = u < u1;
          if (in && !row.whole(u)) x[i] = row.edge(u);
          uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, keep[4], tie[4] = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int e = 0; e < 4; ++e) keep[e] = cutoff.gt(w[e]);
          if (ordered) {
            unsigned some = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              tie[e] = in ? cutoff.eq(w[e]) : 0u;
              some |= tie[e];
            }
            if (__any_sync(0xffffffffu, some != 0u)) {
              unsigned here = 0;
#pragma unroll
              for (int e = 0; e < 4; ++e) here += tie[e] & Compare<DTYPE>::kOnes;
              here = Compare<DTYPE>::total(here);
              unsigned incl = here;
#pragma unroll
              for (int o = 1; o < 32; o <<= 1) {
                const unsigned v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
              }
              unsigned rank_cut = seen + incl - here;
              seen += __shfl_sync(0xffffffffu, incl, 31);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
#pragma unroll
                for (int q = 0; q < VEC / 4; ++q) {   // the word's values in index order
                  const unsigned part = DTYPE == 1 ? 0xffffu << (16 * q) : 0xffffffffu;
                  if (tie[e] & part) {
                    if (rank_cut < cut_eq) keep[e] |= part;
                    ++rank_cut;
                  }
                }
              }
            }
          }
          if (in) {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = (w[e] & keep[e]) | (Compare<DTYPE>::kDropWord & ~keep[e]);
            const uint4 piece = make_uint4(w[0], w[1], w[2], w[3]);
            const int f = row.first(u);
            if (vec && row.whole(u)) {
              __stcs(reinterpret_cast<uint4*>(out + f), piece);
            } else {
              const int c = row.count(u);
#pragma unroll
              for (int e = 0; e < VEC; ++e)
                if (e < c) out[f + e] = Row<DTYPE>::value(piece, e);
            }
          }
        }
      }
    }
    __syncthreads();
    if (tid == 0 && s.token >= 0) p.tokens[r] = s.token;
  } else {
    if (filter) {
      Raw* out = static_cast<Raw*>(p.filtered) + static_cast<long long>(r) * p.filtered_stride;
      const int i0 = row.u0 < row.units ? row.first(row.u0) : p.V, i1 = row.u1 < row.units ? row.first(row.u1) : p.V;
      for (int i = i0 + tid; i < i1; i += NT) out[i] = static_cast<Raw>(DTYPE == 1 ? 0xff80u : 0xff800000u);
    }
    if (tid == 0 && cta == 0) p.tokens[r] = -1;
  }
  if (tid == 0 && cta == 0) {
    if (p.probs) p.probs[r] = prob;
    if (p.kept) p.kept[r] = static_cast<int32_t>(n);
  }
  if (Cl) cluster_sync();   // no CTA leaves while another reads its memory
}

template <int DTYPE, bool Cl>
cudaError_t launch(const SampleParams& p, int ctas, cudaStream_t stream) {
  static std::atomic<unsigned long long> asked{0};   // devices whose limit of shared memory has been raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(asked.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(sample_kernel_row<DTYPE, Cl>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<DTYPE>());
    if (e != cudaSuccess) return e;
    if (dev < 64) asked.fetch_or(1ull << dev);
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(p.R * ctas, 1, 1);
  cfg.blockDim = dim3(Geo<DTYPE>::kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem_bytes<DTYPE>();
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = Cl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, sample_kernel_row<DTYPE, Cl>, p);
}

}  // namespace

cudaError_t launch_sample(int dtype, const SampleParams& p, int sms, cudaStream_t stream) {
  // as many CTAs a row as leave each an SM and 8192 tokens, at most 8.  One row of 128000 bf16: 32 us with one
  // CTA, 30.6 with 2, 28.2 with 4, 27.7 with 8 (adding up the histograms takes 7 of them); 64 rows of
  // 100003 fp32: 130 us with one, 113 with 2.
  int ctas = 1;
  while (ctas < 8 && p.R * ctas * 2 <= sms && p.V >= ctas * 2 * 8192) ctas *= 2;
  if (ctas == 1) return dtype == 1 ? launch<1, false>(p, 1, stream) : launch<0, false>(p, 1, stream);
  return dtype == 1 ? launch<1, true>(p, ctas, stream) : launch<0, true>(p, ctas, stream);
}

}  // namespace sv
