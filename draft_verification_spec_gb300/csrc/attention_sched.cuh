// Work split of the paged attention.
//
// An item is one tile of query rows (the new tokens of a request x the query heads of one key
// head, token-major) of one (request, key head).  It costs a unit per key tile that it has to read, and
// `overhead` units before them (queries in, rows out, the pipeline filled anew).  The units of all
// items, in the order (request, key head, row tile, key tile), are cut into n equal runs, one per CTA,
// whatever the lengths are: a long cache with few rows is split over many CTAs and a short one shares
// a CTA.  (Without the overhead CTAs with many short items ended a third later than the others.)  An
// item that crosses a cut leaves one partial result (maximum, sum, unnormalised rows) per CTA, and the
// combine kernel joins them in the order of the keys, so results do not depend on timing.  Lengths are
// read on the device: the host knows only bounds.
#pragma once

#include "spec_device.cuh"
#include "step_internal.h"

namespace sv {

struct AttnReq {
  int q0, nq;
  int kv;   // keys that the table holds
  int at;   // position of the first new token: counted from the request's length, whatever the table holds
};
// Keys of a request that its row of the table can hold (and that tile arithmetic in 32 bits can).
__device__ __forceinline__ int attn_capacity(const PagedBatch& c) {
  const long long cap = static_cast<long long>(c.table_width) * c.page_size;
  return cap < 0x7fffff00ll ? static_cast<int>(cap) : 0x7fffff00;
}
__device__ __forceinline__ AttnReq attn_request(const PagedBatch& c, int b) {
  AttnReq r;
  r.q0 = min(max(__ldg(c.cu_q + b), 0), c.N);
  r.nq = max(min(__ldg(c.cu_q + b + 1), c.N) - r.q0, 0);
  const int kv = max(__ldg(c.kv_lens + b), 0);
  r.kv = min(kv, attn_capacity(c));
  r.at = kv - r.nq;
  return r;
}

// r / G (G_inv = ceil(2^64 / G), 0 for G = 1): exact for every 32-bit r.
__device__ __forceinline__ int attn_token(const AttnParams& p, int r) {
  return p.G_inv ? static_cast<int>(__umul64hi(static_cast<unsigned long long>(r), p.G_inv)) : r;
}

// A row's factor and lse from its maximum m and sum l (in powers of two).  The sum is zero where the row sees no key, and
// only there: a NaN among its scores makes a NaN of it, which is no mark of an empty row.
__device__ __forceinline__ float attn_factor(float l, float unit) { return l == 0.f ? 0.f : unit / l; }
__device__ __forceinline__ float attn_lse(float m, float l) { return l == 0.f ? ninf() : (m + log2f(l)) * 0.69314718055994531f; }

// Keys [lo, hi) that rows [r0, r1) of the request can see.
__device__ __forceinline__ void attn_keys(const AttnParams& p, const AttnReq& r, int r0, int r1, int* lo, int* hi) {
  *hi = p.causal ? max(min(r.at + attn_token(p, r1 - 1) + 1, r.kv), 0) : r.kv;
  *lo = 0;
  if (p.window > 0) {   // in 64 bits: a position below 0 less a window of 2^31 - 1 does not fit 32
    const long long w = static_cast<long long>(r.at) + attn_token(p, r0) + 1 - p.window;
    *lo = w > 0 ? static_cast<int>(min(w, static_cast<long long>(r.kv))) : 0;
  }
}
// Number of key tiles of row tile t (an item has one at least: its rows are written even where they see no
// key).  They are the first `front` ones, which hold the first tokens that stay visible (SINKS), and those from
// `first` on, where the window begins; the tiles between the two are not looked at.
template <int BN, bool SINKS>
__device__ __forceinline__ int attn_tiles(const AttnParams& p, const AttnReq& r, int t, int bm, int* first, int* front) {
  const int r0 = t * bm, r1 = min(r.nq * p.G, r0 + bm);
  int lo, hi;
  attn_keys(p, r, r0, r1, &lo, &hi);
  *first = lo / BN;
  *front = SINKS ? min((min(p.sinks, hi) + BN - 1) / BN, *first) : 0;
  if (SINKS) return max(*front + max((hi + BN - 1) / BN - *first, 0), 1);
  return max((hi + BN - 1) / BN - *first, 1);
}
__device__ __forceinline__ int attn_row_tiles(const AttnParams& p, const AttnReq& r, int bm) {
  return (r.nq * p.G + bm - 1) / bm;
}
// Units of request b, all key heads; the request's lanes (p.lanes, a power of two: one where a request is
// one row tile) share the row tiles, and every one of them gets the sum.
template <int BN, bool SINKS>
__device__ __forceinline__ long long attn_request_units(const AttnParams& p, int b, int bm) {
  long long n = 0;
  if (b < p.c.B) {
    const AttnReq r = attn_request(p.c, b);
    if (r.nq > 0 && r.at + r.nq > r.kv && blockIdx.x == 0) atomicOr(p.status, kStatusPageRange);   // positions beyond the table
    const int nt = attn_row_tiles(p, r, bm);
    for (int t = threadIdx.x & (p.lanes - 1); t < nt; t += p.lanes) {
      int first, front;
      n += p.overhead + attn_tiles<BN, SINKS>(p, r, t, bm, &first, &front);
    }
  }
  for (int o = p.lanes / 2; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n * p.c.Hkv;
}

struct AttnSplit {
  long long total;   // units of the call
  int n;             // CTAs that share them
  __device__ __forceinline__ long long begin(int c) const { return total * c / n; }
  __device__ __forceinline__ int owner(long long u) const { return static_cast<int>(((u + 1) * n - 1) / total); }
};

// An item, where it starts among the call's units, its key tiles.
struct AttnCursor {
  int b, h, t;
  AttnReq req;
  int first, front, count;
  long long start;
  // Its key tile number j; the first number whose tile is `tile` or behind it.
  template <bool SINKS>
  __device__ __forceinline__ int tile(int j) const {
    return SINKS && j < front ? j : first + j - front;
  }
  template <bool SINKS>
  __device__ __forceinline__ int number(int tile) const {
    if (!SINKS) return tile - first;
    return tile < front ? tile : front + max(tile - first, 0);
  }
  // The key tiles [k0, k1) of the item in the run [begin, end) of a CTA (none if k1 <= k0).
  __device__ __forceinline__ void share(const AttnParams& p, long long begin, long long end, int* k0, int* k1) const {
    const long long t = start + p.overhead;
    *k0 = begin > t ? static_cast<int>(begin - t) : 0;
    *k1 = end - t < count ? static_cast<int>(end - t) : count;
  }
};

template <int THREADS>
struct AttnSchedSmem {
  long long warp[THREADS / 32];
  long long rem, units;
  int b;
};

// Block-wide: the units of the call and how many CTAs share them.
template <int BN, bool SINKS, int THREADS>
__device__ __forceinline__ AttnSplit attn_split(const AttnParams& p, int bm, AttnSchedSmem<THREADS>& s) {
  const int per = THREADS / p.lanes;   // requests at a time (THREADS is a multiple of 32, lanes at most 32)
  long long mine = 0;
  for (int base = 0; base < p.c.B; base += per) {
    const long long n = attn_request_units<BN, SINKS>(p, base + threadIdx.x / p.lanes, bm);
    if ((threadIdx.x & (p.lanes - 1)) == 0) mine += n;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if ((threadIdx.x & 31) == 0) s.warp[threadIdx.x / 32] = mine;
  __syncthreads();
  AttnSplit sp;
  sp.total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) sp.total += s.warp[w];
  const long long n = (sp.total + p.min_units - 1) / p.min_units;
  sp.n = static_cast<int>(n < p.n_max ? n : p.n_max);
  __syncthreads();
  return sp;
}

// Block-wide: the item that unit u belongs to (u < total).
template <int BN, bool SINKS, int THREADS>
__device__ __forceinline__ AttnCursor attn_locate(const AttnParams& p, int bm, long long u, AttnSchedSmem<THREADS>& s) {
  const int lane = threadIdx.x & 31, w = threadIdx.x / 32, per = THREADS / p.lanes;
  long long before = 0;   // units of the requests before this step's
  for (int base = 0; base < p.c.B; base += per) {
    const int b = base + threadIdx.x / p.lanes;
    const long long units = attn_request_units<BN, SINKS>(p, b, bm);
    const long long mine = (threadIdx.x & (p.lanes - 1)) == 0 ? units : 0;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s.warp[w] = incl;
    __syncthreads();
    long long all = 0;
#pragma unroll
    for (int k = 0; k < THREADS / 32; ++k) {
      if (k < w) incl += s.warp[k];
      all += s.warp[k];
    }
    if (u - before >= incl - mine && u - before < incl) {
      s.b = b;
      s.rem = u - before - (incl - mine);
      s.units = units;
    }
    __syncthreads();
    if (u - before < all) break;
    before += all;
  }
  AttnCursor c;
  c.b = s.b;
  c.req = attn_request(p.c, c.b);
  const long long per_head = s.units / p.c.Hkv;
  long long rem = s.rem;
  c.h = static_cast<int>(rem / per_head);
  rem -= per_head * c.h;
  // the row tile: 32 at a time, every warp for itself
  const int nt = attn_row_tiles(p, c.req, bm);
  for (int t0 = 0; t0 < nt; t0 += 32) {
    int first = 0, front = 0;
    const long long mine = t0 + lane < nt ? p.overhead + attn_tiles<BN, SINKS>(p, c.req, t0 + lane, bm, &first, &front) : 0;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, incl > rem);
    if (hit) {
      const int k = __ffs(hit) - 1;
      c.t = t0 + k;
      c.count = static_cast<int>(__shfl_sync(0xffffffffu, mine, k)) - p.overhead;
      c.first = __shfl_sync(0xffffffffu, first, k);
      c.front = SINKS ? __shfl_sync(0xffffffffu, front, k) : 0;
      c.start = u - (rem - __shfl_sync(0xffffffffu, incl - mine, k));
      break;
    }
    rem -= __shfl_sync(0xffffffffu, incl, 31);
  }
  __syncthreads();
  return c;
}

// One thread of every CTA, at its last item (`later`: it is not the CTA's first) or, without work (or not
// yet done), with cur = null: leaves the record for the combine kernel, an empty one for null.
__device__ __forceinline__ void attn_leave_join(const AttnParams& p, const AttnSplit& sp, int cta, int bm, const AttnCursor* cur,
                                                bool later) {
  AttnJoin j = {};
  if (cur) {
    int k0, k1;
    cur->share(p, sp.begin(cta), sp.begin(cta + 1), &k0, &k1);
    if (k0 == 0 && k1 < cur->count) {
      j.row0 = cur->t * bm;
      j.rows = min(cur->req.nq * p.G - j.row0, bm);
      j.token0 = cur->req.q0;
      j.head0 = cur->h * p.G;
      j.last = sp.owner(cur->start + p.overhead + cur->count - 1);
      j.slot = 2 * cta + (later ? 1 : 0);
    }
  }
  p.joins[cta] = j;
}

// The next item with key tiles in a run that ends at `end`; false if there is none.
template <int BN, bool SINKS>
__device__ __forceinline__ bool attn_next(const AttnParams& p, int bm, long long end, AttnCursor* c) {
  c->start += p.overhead + c->count;
  if (c->start + p.overhead >= end) return false;
  if (++c->t >= attn_row_tiles(p, c->req, bm)) {
    c->t = 0;
    if (++c->h == p.c.Hkv) {
      c->h = 0;
      do {
        c->req = attn_request(p.c, ++c->b);
      } while (c->req.nq == 0);
    }
  }
  c->count = attn_tiles<BN, SINKS>(p, c->req, c->t, bm, &c->first, &c->front);
  return true;
}

}  // namespace sv
