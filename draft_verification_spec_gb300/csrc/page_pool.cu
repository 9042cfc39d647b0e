// The pages of a paged cache: which request holds which (assign, compact), and the copies that follow in every array of
// the pool.
//
// Assigning: row b of the new table holds the pages of lens[b] tokens.  It inherits the first kept[b] tokens' pages from
// row parents[b] of the old one.  Whole pages are shared by all that inherit them; the page that ends inside
// (kept % page_size) will be written to, so of those that inherit it one alone keeps it: nobody if some row only reads
// it, else the lowest row; the others get a fresh page and a copy.  All further pages are fresh.  Fresh pages are the
// lowest ids that nobody inherits, in the order (row, column); what nobody inherits is free, so nothing is released by name.
// Compacting: of u used pages those with ids >= u, in rising order, move to the unused ids below u, in rising order.
//
// Both are one cluster of CTAs over the table and one mark a page, with cluster barriers between the phases: the marks
// (4 bytes a page) and the tables stay in L2, and a phase is a pass over one of them.  Every result is a minimum or a
// rank, so it depends on no timing.  Bound: latency of the passes (launch and barriers where the pool is small).
// The copies are a second kernel (programmatic dependent launch) that reads the moves: bound by HBM, a page's bytes
// read and written once for every array.
// Measured: 64 requests of up to 16384 tokens in pages of 16 (a table of 64 x 1026, 50,329 pages) between two steps 18 us on
// the device + 3 for the copies' empty grid; 8 prompts forked into 64 samples, 56 pages copied in 32 arrays (118 MB) 14 +
// 16; a pool of 8997 pages moved together, 2.26 GB in 8 arrays, 17 + 337 (6.7 TB/s).  Rows looked up once a CTA and table entries
// four in flight brought the first from 24 us.
#include <climits>

#include "spec_async.cuh"
#include "step_internal.h"

namespace sv {

namespace {

constexpr int kPlanThreads = 1024, kCopyThreads = 256;
constexpr int kCopyBytes = kCopyThreads * 16 * 4;   // bytes of a page that a CTA copies at a time
constexpr int kCols = 128;                      // columns of a row that a warp has in flight

__device__ __forceinline__ int block_sum(int v, int* s) {
  v = warp_sum_int(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x / 32] = v;
  __syncthreads();
  int all = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) all += s[w];
  return all;
}
// Sum of v over the threads before this one; *all: over all.
__device__ __forceinline__ int block_before(int v, int* s, int* all) {
  const int lane = threadIdx.x & 31;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  __syncthreads();
  if (lane == 31) s[threadIdx.x / 32] = incl;
  __syncthreads();
  int before = incl - v, total = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < static_cast<int>(threadIdx.x / 32)) before += s[w];
    total += s[w];
  }
  *all = total;
  return before;
}

struct Row {
  int need, full, part, parent;   // pages of the new row; inherited: whole pages, one that ends inside, from whom
};
__device__ __forceinline__ Row row_of(const PageParams& p, int b) {
  Row r;
  int n = max(__ldg(p.lens + b), 0);
  const long long cap = static_cast<long long>(p.width) * p.page_size;
  if (n > cap) {   // more tokens than the row has columns for
    n = static_cast<int>(cap);
    atomicOr(p.status, kStatusPageRange);
  }
  r.parent = p.parents ? __ldg(p.parents + b) : b;
  const bool has = r.parent >= 0 && r.parent < p.rows;
  const int k = has ? min(max(__ldg(p.kept + b), 0), n) : 0;
  if (!has) r.parent = 0;
  r.need = n / p.page_size + (n % p.page_size > 0);
  r.full = k / p.page_size;
  r.part = k % p.page_size > 0;
  return r;
}
// Items of the table, a warp each: `cols` columns of a row, as many as give every warp one (and 512 at most).
struct Items {
  int cols, chunks, n;
};
__device__ __forceinline__ Items items_of(const PageParams& p, int warps) {
  Items it;
  const long long per = (static_cast<long long>(p.rows) * p.width + warps - 1) / warps;
  it.cols = static_cast<int>(min(max((per + kCols - 1) / kCols * kCols, static_cast<long long>(kCols)), 512ll));
  it.chunks = (p.width + it.cols - 1) / it.cols;
  it.n = p.rows * it.chunks;
  return it;
}
__device__ __forceinline__ int entry(const PageParams& p, int b, int j) { return __ldg(p.table + b * p.stride + j); }
__device__ __forceinline__ bool valid(const PageParams& p, int pg) { return pg >= 0 && pg < p.pages; }

// This CTA's share [first, last) of the pages.
__device__ __forceinline__ void share_of(const PageParams& p, int rank, int n, int* first, int* last) {
  *first = static_cast<int>(static_cast<long long>(p.pages) * rank / n);
  *last = static_cast<int>(static_cast<long long>(p.pages) * (rank + 1) / n);
}
__device__ __forceinline__ void clear_marks(const PageParams& p, int rank, int n, int to) {
  int first, last;
  share_of(p, rank, n, &first, &last);
  for (int i = first + threadIdx.x; i < last; i += kPlanThreads) __stcg(p.mark + i, to);
}

__global__ void __launch_bounds__(kPlanThreads, 1) assign_pages_kernel(const PageParams p) {
  __shared__ int s_sum[kPlanThreads / 32];
  __shared__ Row s_rows[kPlanThreads];   // the first rows, looked up once
  asm volatile("griddepcontrol.launch_dependents;");
  const int rank = cluster_rank(), n = cluster_ncta(), tid = threadIdx.x, lane = tid & 31;
  const int warp = rank * (kPlanThreads / 32) + tid / 32, warps = n * (kPlanThreads / 32);
  const Items items = items_of(p, warps);
  int first, last;
  share_of(p, rank, n, &first, &last);

  if (tid < p.rows) s_rows[tid] = row_of(p, tid);
  clear_marks(p, rank, n, INT_MAX);
  __syncthreads();
  auto row = [&](int b) { return b < kPlanThreads ? s_rows[b] : row_of(p, b); };
  cluster_sync();
  // marks: -1 for a page that some row only reads, else the lowest row that will write to it
  for (int it = warp; it < items.n; it += warps) {
    const int b = it / items.chunks, first_col = (it - b * items.chunks) * items.cols;
    const Row r = row(b);
    const int end = min(min(r.full + r.part, p.width), first_col + items.cols);
    for (int j0 = first_col; j0 < end; j0 += kCols) {
      int pg[kCols / 32];
#pragma unroll
      for (int i = 0; i < kCols / 32; ++i) {
        const int j = j0 + i * 32 + lane;
        pg[i] = j < end ? entry(p, r.parent, j) : -1;
      }
#pragma unroll
      for (int i = 0; i < kCols / 32; ++i) {
        const int j = j0 + i * 32 + lane;
        if (j >= end) continue;
        if (valid(p, pg[i]))
          atomicMin(p.mark + pg[i], j < r.full ? -1 : b);
        else
          atomicOr(p.status, kStatusPageRange);
      }
    }
  }
  cluster_sync();
  // free pages of this CTA's share; the first CTA: how many fresh pages the rows before each one take
  int count = 0;
  for (int i = first + tid; i < last; i += kPlanThreads) count += __ldcg(p.mark + i) == INT_MAX;
  count = block_sum(count, s_sum);
  if (tid == 0) __stcg(p.counts + rank, count);
  if (rank == 0) {
    int base = 0;
    for (int b0 = 0; b0 < p.rows; b0 += kPlanThreads) {
      const int b = b0 + tid;
      int fresh = 0, keep = 0, from = -1;   // fresh pages, columns that stay, the page that is copied
      Row r = {0, 0, 0, 0};
      if (b < p.rows) {
        r = row(b);
        keep = r.full;
        if (r.part) {
          const int pg = entry(p, r.parent, r.full);
          if (!valid(p, pg) || __ldcg(p.mark + pg) == b)
            ++keep;
          else
            from = pg;
        }
        fresh = r.need - keep;
      }
      int all;
      const int before = block_before(fresh, s_sum, &all);
      if (b < p.rows) {
        __stcg(p.plan + b, make_int4(r.parent, keep, r.need, base + before));
        __stcg(p.src + b, from);
      }
      base += all;
    }
    if (tid == 0) __stcg(p.wanted, base);
  }
  cluster_sync();
  // the free pages in rising order, as many as are wanted
  const int wanted = __ldcg(p.wanted);
  int base = 0, there = 0;
  for (int c = 0; c < n; ++c) {
    const int k = __ldcg(p.counts + c);
    if (c < rank) base += k;
    there += k;
  }
  if (rank == 0 && tid == 0 && there < wanted) atomicOr(p.status, kStatusPageRange);
  for (int i0 = first; i0 < last && base < wanted; i0 += kPlanThreads) {
    const int i = i0 + tid, is = i < last && __ldcg(p.mark + i) == INT_MAX;
    int all;
    const int at = base + block_before(is, s_sum, &all);
    if (is && at < wanted) __stcg(p.list + at, i);
    base += all;
  }
  cluster_sync();
  // the new table and the copies
  for (int it = warp; it < items.n; it += warps) {
    const int b = it / items.chunks, first_col = (it - b * items.chunks) * items.cols;
    const int4 r = __ldcg(p.plan + b);   // parent, columns that stay, columns, place of the first fresh page
    const int from = first_col == 0 && lane == 0 ? __ldcg(p.src + b) : -1;
    auto fresh_page = [&](int j) { return r.w + j - r.y < there ? __ldcg(p.list + r.w + j - r.y) : -1; };
    const int end = min(p.width, first_col + items.cols);
    for (int j0 = first_col; j0 < end; j0 += kCols) {
      int to[kCols / 32];
#pragma unroll
      for (int i = 0; i < kCols / 32; ++i) {
        const int j = j0 + i * 32 + lane;
        to[i] = -1;
        if (j < end && j < r.y)
          to[i] = entry(p, r.x, j);
        else if (j < end && j < r.z)
          to[i] = fresh_page(j);
      }
#pragma unroll
      for (int i = 0; i < kCols / 32; ++i) {
        const int j = j0 + i * 32 + lane;
        if (j < end) p.out[b * p.out_stride + j] = valid(p, to[i]) ? to[i] : -1;
      }
    }
    if (from >= 0) {   // the first fresh page is its copy
      const int dst = fresh_page(r.y);
      __stcg(p.dst + b, dst);
      if (dst < 0) __stcg(p.src + b, -1);
    }
  }
  if (rank == 0 && tid == 0) __stcg(p.moves, p.rows);
}

__global__ void __launch_bounds__(kPlanThreads, 1) compact_pages_kernel(const PageParams p) {
  __shared__ int s_sum[kPlanThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;");
  const int rank = cluster_rank(), n = cluster_ncta(), tid = threadIdx.x, lane = tid & 31;
  const int warp = rank * (kPlanThreads / 32) + tid / 32, warps = n * (kPlanThreads / 32);
  const Items items = items_of(p, warps);
  int first, last;
  share_of(p, rank, n, &first, &last);

  clear_marks(p, rank, n, 0);
  cluster_sync();
  for (int it = warp; it < items.n; it += warps) {
    const int b = it / items.chunks, first_col = (it - b * items.chunks) * items.cols;
    const int end = min(p.width, first_col + items.cols);
    for (int j0 = first_col; j0 < end; j0 += kCols) {
      int pg[kCols / 32];
#pragma unroll
      for (int i = 0; i < kCols / 32; ++i) pg[i] = j0 + i * 32 + lane < end ? entry(p, b, j0 + i * 32 + lane) : -1;
#pragma unroll
      for (int i = 0; i < kCols / 32; ++i) {
        if (valid(p, pg[i]))
          __stcg(p.mark + pg[i], 1);
        else if (pg[i] != -1)
          atomicOr(p.status, kStatusPageRange);
      }
    }
  }
  cluster_sync();
  int count = 0;
  for (int i = first + tid; i < last; i += kPlanThreads) count += __ldcg(p.mark + i);
  count = block_sum(count, s_sum);
  if (tid == 0) __stcg(p.counts + rank, count);
  cluster_sync();
  int base = 0, used = 0;   // used pages before this CTA's share, in all
  for (int c = 0; c < n; ++c) {
    const int k = __ldcg(p.counts + c);
    if (c < rank) base += k;
    used += k;
  }
  int below = 0;            // used pages below `used`: they stay
  {
    int c = 0, c_first = 0, c_last = 0;
    for (;; ++c) {          // the share that `used` lies in (or ends at)
      share_of(p, c, n, &c_first, &c_last);
      if (used <= c_last || c == n - 1) break;
      below += __ldcg(p.counts + c);
    }
    int k = 0;
    for (int i = c_first + tid; i < used; i += kPlanThreads) k += __ldcg(p.mark + i);
    below += block_sum(k, s_sum);
  }
  for (int i0 = first; i0 < last; i0 += kPlanThreads) {
    const int i = i0 + tid, is = i < last ? __ldcg(p.mark + i) : 0;
    int all;
    const int before = base + block_before(is, s_sum, &all);   // used pages before page i
    if (i < last && is && i >= used) __stcg(p.src + before - below, i);
    if (i < last && !is && i < used) __stcg(p.dst + i - before, i);
    base += all;
  }
  cluster_sync();
  const int moves = used - below;
  for (int i = rank * kPlanThreads + tid; i < moves; i += n * kPlanThreads) __stcg(p.mark + __ldcg(p.src + i), -1 - __ldcg(p.dst + i));
  if (rank == 0 && tid == 0) {
    __stcg(p.moves, moves);
    *p.used = used;
  }
  cluster_sync();
  for (int it = warp; it < items.n; it += warps) {
    const int b = it / items.chunks, first_col = (it - b * items.chunks) * items.cols;
    const int end = min(p.width, first_col + items.cols);
    for (int j0 = first_col; j0 < end; j0 += kCols) {
      int pg[kCols / 32], to[kCols / 32];
#pragma unroll
      for (int i = 0; i < kCols / 32; ++i) pg[i] = j0 + i * 32 + lane < end ? entry(p, b, j0 + i * 32 + lane) : -1;
#pragma unroll
      for (int i = 0; i < kCols / 32; ++i) to[i] = valid(p, pg[i]) ? __ldcg(p.mark + pg[i]) : 0;
#pragma unroll
      for (int i = 0; i < kCols / 32; ++i) {
        const int j = j0 + i * 32 + lane;
        if (j < end) p.out[b * p.out_stride + j] = !valid(p, pg[i]) ? -1 : to[i] < 0 ? -1 - to[i] : pg[i];
      }
    }
  }
}

template <typename V>
__device__ __forceinline__ void copy_bytes(const uint8_t* src, uint8_t* dst, int bytes) {
  const int n = bytes / static_cast<int>(sizeof(V));
  const V* s = reinterpret_cast<const V*>(src);
  V* d = reinterpret_cast<V*>(dst);
  for (int i = threadIdx.x; i < n; i += kCopyThreads * 4) {
    V x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k * kCopyThreads < n) x[k] = s[i + k * kCopyThreads];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k * kCopyThreads < n) d[i + k * kCopyThreads] = x[k];
  }
}

// A CTA a chunk of a page in an array at a time, chunks innermost.
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const PageParams p, int chunks) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long per = static_cast<long long>(p.n_arrays) * chunks, items = __ldcg(p.moves) * per;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int m = static_cast<int>(it / per);
    const long long in = it - m * per;   // array and chunk
    const int a = static_cast<int>(in / chunks);
    const int src = __ldcg(p.src + m), dst = __ldcg(p.dst + m);
    if (src < 0) continue;
    const PageArray arr = p.arrays[a];
    const long long from = (in - static_cast<long long>(a) * chunks) * kCopyBytes;
    const int bytes = static_cast<int>(min(arr.bytes - from, static_cast<long long>(kCopyBytes)));
    if (bytes <= 0) continue;
    const uint8_t* s = arr.base + src * arr.stride + from;
    uint8_t* d = arr.base + dst * arr.stride + from;
    const unsigned low = (static_cast<unsigned>(reinterpret_cast<uintptr_t>(arr.base)) | static_cast<unsigned>(arr.stride) |
                          static_cast<unsigned>(arr.bytes)) & 15u;
    if (low == 0)
      copy_bytes<uint4>(s, d, bytes);
    else if ((low & 3) == 0)
      copy_bytes<uint32_t>(s, d, bytes);
    else
      copy_bytes<uint8_t>(s, d, bytes);
  }
}

}  // namespace

cudaError_t launch_pages(bool compact, const PageParams& p, long long max_bytes, int sms, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 8;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(8, 1, 1);
  cfg.blockDim = dim3(kPlanThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = compact ? cudaLaunchKernelEx(&cfg, compact_pages_kernel, p) : cudaLaunchKernelEx(&cfg, assign_pages_kernel, p);
  if (e != cudaSuccess || p.n_arrays == 0 || max_bytes == 0) return e;
  const int chunks = static_cast<int>((max_bytes + kCopyBytes - 1) / kCopyBytes);
  const long long most = static_cast<long long>(compact ? p.pages / 2 : p.rows) * p.n_arrays * chunks;
  const long long grid = most < 8ll * sms ? most : 8ll * sms;
  if (grid == 0) return cudaSuccess;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kCopyThreads, 1, 1);
  return cudaLaunchKernelEx(&cfg, copy_pages_kernel, p, chunks);
}

}  // namespace sv
