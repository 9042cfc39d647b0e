// Attention of new tokens over a paged cache, tcgen05 kernel: 256-row tiles, pages that TMA can copy.
//
// One CTA per SM works through its run of (item, key tile) units.  A tile's 256 rows are two halves
// of 128 (the M of one MMA) that share every key tile of 128 keys.  Ten warps:
//   0-3, 4-7  softmax of half 0 and 1: a thread owns a row (TMEM lane): reads the row's 128 scores,
//             keeps the running maximum and sum, writes the probabilities back over the scores as
//             the second MMA's A operand, and rescales O in TMEM;
//   8         TMA producer: one box per page, head and 64 dims, 128-byte swizzle;
//   9         MMA issuer: S = Q K^T (both operands in shared memory) and O += P V (P in TMEM).
// The two halves alternate: while one half's softmax runs, the tensor core works on the other's.
// TMEM (512 columns): S0 | S1 | O0 | O1, P_i in S_i's columns.
//
// O is rescaled only when a row's maximum grows by more than 2^8 over the reference its exponentials
// use; until then the probabilities may reach 2^8, which neither type overflows and the final division
// by the sum undoes.  S(j) is committed after P V(j-1) of the same half in issue order, so a softmax
// thread that has seen S(j) may touch O.
//
// Keys at or beyond the item's last one: pages that lie wholly there are read at an out-of-range page
// coordinate, which TMA fills with zeros; the rest of the last page can hold anything, so its value
// rows are zeroed in shared memory before the MMA reads them (0 x NaN would be NaN); scores are
// selected, not multiplied.
//
// Every wait is bounded: after `wait_limit` the kernel sets the status word, drains its copies and
// MMAs, frees TMEM and returns.
#pragma once

#include <cuda.h>

#include "attention_mma.cuh"
#include "spec_async.cuh"

namespace sv {

constexpr int kTcThreads = 320;
constexpr int kTcBN = 128, kTcBM = 256;

template <int DP>
struct AttnTcGeom {
  static constexpr int kTile = 128 * DP * 2;                 // one half's Q, one tile's K or V
  static constexpr int kKStages = DP == 64 ? 4 : 3, kVStages = DP == 64 ? 4 : 2;
  static constexpr int kSmem = 1024 + (2 + kKStages + kVStages) * kTile;
};

struct AttnTcBars {
  unsigned long long k_full[4], k_empty[4], v_full[4], v_empty[4], s_full[2], p_full[2], o_full[2], q_full[2], drain;
};

// ------------------------------------------------------------------------------------ PTX wrappers
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// 32 consecutive columns of this thread's TMEM lane.
__device__ __forceinline__ void tc_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int d, int token, int head, int page,
                                        uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(d), "r"(token), "r"(head), "r"(page), "r"(bar)
      : "memory");
}
// Shared-memory operand with the 128-byte swizzle.  K-major: rows of 128 bytes, 8-row groups 1024 bytes
// apart (the leading offset is not used).  MN-major: 64-value blocks `lead` bytes apart, groups of 8
// k-rows 1024 bytes apart.
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t lead) {
  return static_cast<uint64_t>((addr >> 4) & 0x3fffu) | (static_cast<uint64_t>(lead >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

struct TcWait {
  volatile int* abort;
  long long limit;
  int32_t* status;
  // Waits for the phase; false once the limit has passed or another warp gave up.
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
    if (mbar_try(bar, parity)) return true;
    const unsigned long long t0 = global_ns();
    while (true) {
#pragma unroll 1
      for (int k = 0; k < 16; ++k)
        if (mbar_try(bar, parity)) return true;
      if (*abort) return false;
      if (static_cast<long long>(global_ns() - t0) > limit) {
        *abort = 1;
        atomicOr(status, kStatusTimeout);
        return false;
      }
    }
  }
};

template <bool BF16, int DP>
__global__ void __launch_bounds__(kTcThreads, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const AttnParams p) {
  using A = AttnType<BF16>;
  using Geo = AttnTcGeom<DP>;
  constexpr int BM = kTcBM, BN = kTcBN, SUB = DP / 64, KST = Geo::kKStages, VST = Geo::kVStages, TILE = Geo::kTile;
  extern __shared__ uint8_t smem_raw[];
  __shared__ AttnSchedSmem<kTcThreads> sched;
  __shared__ __align__(8) AttnTcBars bars;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t s_q = base, s_k = base + 2 * TILE, s_v = s_k + KST * TILE;

  const AttnSplit split = attn_split<BN>(p, BM, sched);
  const int cta = blockIdx.x;
  asm volatile("griddepcontrol.launch_dependents;");
  if (cta >= split.n) return;
  const long long u_begin = split.begin(cta), u_end = split.begin(cta + 1);
  AttnCursor cur = attn_locate<BN>(p, BM, u_begin, sched);

  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_addr(&bars.k_full[i]), 1);
      mbar_init(smem_addr(&bars.k_empty[i]), 1);
      mbar_init(smem_addr(&bars.v_full[i]), 1);
      mbar_init(smem_addr(&bars.v_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&bars.s_full[i]), 1);
      mbar_init(smem_addr(&bars.p_full[i]), 128);
      mbar_init(smem_addr(&bars.o_full[i]), 1);
      mbar_init(smem_addr(&bars.q_full[i]), 128);
    }
    mbar_init(smem_addr(&bars.drain), 1);
    mbar_fence_init();
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&s_tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const TcWait wait{&s_abort, p.wait_limit, p.status};
  long long u = u_begin;

  if (warp == 8) {
    // ------------------------------------------------------------------------------ TMA producer
    const int P = p.c.page_size, rows = min(P, BN), boxes = BN / rows;   // boxes of 64 dims per tile
    unsigned g = 0;                                                      // key tiles of this CTA so far
    bool ok = true;
    while (ok) {
      const int kt0 = cur.first + cur.at;
      const int len = static_cast<int>(min(static_cast<long long>(cur.count - cur.at), u_end - u));
      const int r0 = cur.t * BM, r1 = min(cur.req.nq * p.G, r0 + BM);
      int lo, hi;
      attn_keys(p, cur.req, r0, r1, &lo, &hi);
      const int32_t* table = p.c.table + static_cast<long long>(cur.b) * p.c.table_stride;
      for (int j = 0; ok && j < len; ++j, ++g) {
        // this lane's boxes: page `i` of the tile (i = lane: at most 16 pages of 8 tokens and more)
        const int key = (kt0 + j) * BN + lane * rows;
        int pg = p.c.pages;   // out of range: zeros
        if (lane < boxes && key < hi) {
          pg = __ldg(table + key / P);
          if (pg < 0 || pg >= p.c.pages) {
            atomicOr(p.status, kStatusPageRange);
            pg = p.c.pages;
          }
        }
        const int tok = key % P;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
          const int st = which ? g % VST : g % KST;
          const uint32_t ph = which ? (g / VST) & 1 : (g / KST) & 1;
          const uint32_t full = smem_addr(which ? &bars.v_full[st] : &bars.k_full[st]);
          const uint32_t empty = smem_addr(which ? &bars.v_empty[st] : &bars.k_empty[st]);
          ok = __all_sync(0xffffffffu, ok && wait(empty, ph ^ 1));
          if (!ok) break;
          if (lane == 0) mbar_arrive_tx(full, TILE);
          __syncwarp();
          if (lane < boxes) {
            const uint32_t dst = (which ? s_v : s_k) + st * TILE + lane * rows * 128;
#pragma unroll
            for (int s = 0; s < SUB; ++s) tma_box(dst + s * 128 * 128, which ? &map_v : &map_k, s * 64, tok, cur.h, pg, full);
          }
          __syncwarp();
        }
      }
      u += len;
      if (u >= u_end) break;
      attn_next<BN>(p, BM, &cur);
    }
    if (!ok) {
      // gave up: the copies in flight still land before the block's memory is given back
      for (unsigned i = g > 4 ? g - 4 : 0; i <= g; ++i) {
        const unsigned long long t0 = global_ns();
        while (!(mbar_try(smem_addr(&bars.k_full[i % KST]), (i / KST) & 1) && mbar_try(smem_addr(&bars.v_full[i % VST]), (i / VST) & 1)) &&
               global_ns() - t0 < 20000000ull) {
        }
      }
    }
  } else if (warp == 9) {
    // -------------------------------------------------------------------------------- MMA issuer
    constexpr uint32_t kType = BF16 ? 1u : 0u;
    constexpr uint32_t kCommon = (1u << 4) | (kType << 7) | (kType << 10) | ((128u >> 4) << 24);
    constexpr uint32_t kIdescS = kCommon | ((128u >> 3) << 17);
    constexpr uint32_t kIdescO = kCommon | (1u << 16) | ((static_cast<uint32_t>(DP) >> 3) << 17);
    unsigned g = 0, nh_tiles[2] = {0, 0}, segs[2] = {0, 0};
    bool ok = true;
    auto issue_s = [&](int half, int st) {
#pragma unroll
      for (int k = 0; k < DP / 16; ++k) {
        const uint32_t off = (k / 4) * 16384 + (k % 4) * 32;
        tc_mma_ss(tmem + half * 128, tc_desc(s_q + half * TILE + off, 16), tc_desc(s_k + st * TILE + off, 16), kIdescS, k > 0);
      }
    };
    auto issue_o = [&](int half, int st, bool acc) {
#pragma unroll
      for (int k = 0; k < BN / 16; ++k)
        tc_mma_ts(tmem + 256 + half * 128, tmem + half * 128 + k * 8, tc_desc(s_v + st * TILE + k * 2048, 16384), kIdescO,
                  acc || k > 0);
    };
    while (ok) {
      const int kt0 = cur.first + cur.at;
      const int len = static_cast<int>(min(static_cast<long long>(cur.count - cur.at), u_end - u));
      const int r0 = cur.t * BM, r1 = min(cur.req.nq * p.G, r0 + BM);
      const int nh = r1 - r0 > 128 ? 2 : 1;
      int lo, hi;
      attn_keys(p, cur.req, r0, r1, &lo, &hi);
      for (int h = 0; ok && h < nh; ++h) ok = __all_sync(0xffffffffu, wait(smem_addr(&bars.q_full[h]), segs[h]++ & 1));
      if (ok) ok = __all_sync(0xffffffffu, wait(smem_addr(&bars.k_full[g % KST]), (g / KST) & 1));
      if (!ok) break;
      tc_fence_after();
      if (lane == 0) {
        for (int h = 0; h < nh; ++h) {
          issue_s(h, g % KST);
          tc_commit(smem_addr(&bars.s_full[h]));
        }
        tc_commit(smem_addr(&bars.k_empty[g % KST]));
      }
      __syncwarp();
      for (int j = 0; j < len; ++j, ++g) {
        const int vst = g % VST, kn = (g + 1) % KST;
        ok = __all_sync(0xffffffffu, wait(smem_addr(&bars.v_full[vst]), (g / VST) & 1));
        if (!ok) break;
        const int valid = hi - (kt0 + j) * BN;
        if (valid < BN) {   // the item's last key tile: value rows that are not its own become zero
          for (int i = max(valid, 0) * 8 + lane; i < BN * 8; i += 32)
#pragma unroll
            for (int s = 0; s < SUB; ++s)
              asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(s_v + vst * TILE + s * 16384 + i * 16), "r"(0u) : "memory");
          fence_async_smem();
          __syncwarp();
        }
        for (int h = 0; h < nh; ++h) {
          ok = __all_sync(0xffffffffu, wait(smem_addr(&bars.p_full[h]), nh_tiles[h] & 1));
          if (!ok) break;
          ++nh_tiles[h];
          tc_fence_after();
          if (lane == 0) {
            issue_o(h, vst, j > 0);
            if (j + 1 == len) tc_commit(smem_addr(&bars.o_full[h]));
            if (h + 1 == nh) tc_commit(smem_addr(&bars.v_empty[vst]));
          }
          __syncwarp();
          if (j + 1 < len) {
            if (h == 0) {
              ok = __all_sync(0xffffffffu, wait(smem_addr(&bars.k_full[kn]), ((g + 1) / KST) & 1));
              if (!ok) break;
              tc_fence_after();
            }
            if (lane == 0) {
              issue_s(h, kn);
              tc_commit(smem_addr(&bars.s_full[h]));
              if (h + 1 == nh) tc_commit(smem_addr(&bars.k_empty[kn]));
            }
            __syncwarp();
          }
        }
        if (!ok) break;
      }
      u += len;
      if (!ok || u >= u_end) break;
      attn_next<BN>(p, BM, &cur);
    }
    if (!ok) {   // gave up: the MMAs in flight finish before TMEM is freed
      if (lane == 0) tc_commit(smem_addr(&bars.drain));
      const unsigned long long t0 = global_ns();
      while (!mbar_try(smem_addr(&bars.drain), 0) && global_ns() - t0 < 100000000ull) {
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------------------------------ softmax
    const int half = warp >> 2, row = tid & 127;   // row of the half = TMEM lane
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + half * 128, t_o = tmem + lanes + 256 + half * 128;
    const uint32_t bar_s = smem_addr(&bars.s_full[half]), bar_p = smem_addr(&bars.p_full[half]);
    unsigned tiles = 0, segs = 0;
    bool ok = true;
    while (ok) {
      const int kt0 = cur.first + cur.at;
      const int len = static_cast<int>(min(static_cast<long long>(cur.count - cur.at), u_end - u));
      const int r0 = cur.t * BM, r1 = min(cur.req.nq * p.G, r0 + BM);
      if (r1 - r0 > half * 128) {
        const int r = r0 + half * 128 + row;
        const bool mine = r < r1;
        const bool busy = r0 + half * 128 + (warp & 3) * 32 < r1;   // some row of this warp exists
        {
          const int tok = cur.req.q0 + r / p.G, head = cur.h * p.G + r % p.G;
          const uint8_t* src = p.q + (tok * p.q_token + head * p.q_head) * 2;
          const uint32_t dst = s_q + half * TILE + row * 128;
#pragma unroll
          for (int c = 0; c < DP / 8; ++c) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (mine && c * 8 < p.c.D) v = __ldg(reinterpret_cast<const uint4*>(src + c * 16));
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst + (c / 8) * 16384 + (((c & 7) ^ (row & 7)) << 4)),
                         "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                         : "memory");
          }
          fence_async_smem();
          mbar_arrive(smem_addr(&bars.q_full[half]));
        }
        int row_lo = 0, row_hi = 0;
        if (mine) attn_keys(p, cur.req, r, r + 1, &row_lo, &row_hi);
        // key tiles in [free_lo, free_hi) need no mask for any row of the warp
        const int w_hi = __reduce_min_sync(0xffffffffu, mine ? row_hi : 0x7fffffff);
        const int w_lo = __reduce_max_sync(0xffffffffu, mine ? row_lo : 0);
        float m = ninf(), l = 0.f;
        for (int j = 0; j < len; ++j, ++tiles) {
          ok = __all_sync(0xffffffffu, wait(bar_s, tiles & 1));
          if (!ok) break;
          tc_fence_after();
          if (busy) {
            uint32_t s[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) tc_ld32(t_s + c * 32, s + c * 32);
            tc_wait_ld();
            const int k0 = (kt0 + j) * BN;
            if (k0 + BN > w_hi || k0 < w_lo) {
              const int a = row_lo - k0, b = row_hi - k0;
#pragma unroll
              for (int i = 0; i < 128; ++i) s[i] = i >= a && i < b ? s[i] : 0xff800000u;
            }
            float t[4] = {ninf(), ninf(), ninf(), ninf()};
#pragma unroll
            for (int i = 0; i < 128; i += 8)
#pragma unroll
              for (int c = 0; c < 4; ++c)
                t[c] = fmaxf(fmaxf(t[c], __uint_as_float(s[i + c])), __uint_as_float(s[i + c + 4]));
            // in units of the scaled scores (the scale is positive)
            const float top = fmaxf(m, fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * p.scale_log2);
            const bool grow = top - m > 8.f || (m == ninf() && top > m);
            if (__any_sync(0xffffffffu, grow)) {
              const float ref = top == ninf() ? 0.f : top;
              const float f = ex2(m - ref);
              l *= f;
              m = top;
              if (j > 0) {
#pragma unroll 1
                for (int c = 0; c < DP / 32; ++c) {
                  uint32_t o[32];
                  tc_ld32(t_o + c * 32, o);
                  tc_wait_ld();
#pragma unroll
                  for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                  tc_st32(t_o + c * 32, o);
                }
              }
            }
            const float ref = m == ninf() ? 0.f : m;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t pk[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float x = ex2(fmaf(__uint_as_float(s[c * 64 + 2 * i]), p.scale_log2, -ref));
                const float y = ex2(fmaf(__uint_as_float(s[c * 64 + 2 * i + 1]), p.scale_log2, -ref));
                sum[(2 * i) & 3] += x;
                sum[(2 * i + 1) & 3] += y;
                pk[i] = A::pack(x, y);
              }
              tc_st32(t_s + c * 32, pk);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tc_wait_st();
          }
          tc_fence_before();
          mbar_arrive(bar_p);
        }
        if (!ok) break;
        ok = __all_sync(0xffffffffu, wait(smem_addr(&bars.o_full[half]), segs & 1));
        ++segs;
        if (!ok) break;
        tc_fence_after();
        const bool whole = len == cur.count;
        const float inv = whole ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
        const long long tok = cur.req.q0 + r / p.G;
        const long long orow = tok * p.Hq + cur.h * p.G + r % p.G;
        const long long prow = static_cast<long long>(2 * cta + (u == u_begin ? 0 : 1)) * BM + half * 128 + row;
        if (busy) {
#pragma unroll 1
          for (int c = 0; c < DP / 32; ++c) {
            uint32_t o[32];
            __syncwarp();
            tc_ld32(t_o + c * 32, o);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              const int d = c * 32 + i;
              if (!mine || d >= p.c.D) continue;
              float f[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(o[i + e]) * inv;
              if (whole) {
                *reinterpret_cast<uint4*>(p.out + (orow * p.c.D + d) * 2) =
                    make_uint4(A::pack(f[0], f[1]), A::pack(f[2], f[3]), A::pack(f[4], f[5]), A::pack(f[6], f[7]));
              } else {
                float4* dst = reinterpret_cast<float4*>(p.part_o + prow * p.c.D + d);
                dst[0] = make_float4(f[0], f[1], f[2], f[3]);
                dst[1] = make_float4(f[4], f[5], f[6], f[7]);
              }
            }
          }
        }
        if (mine) {
          if (!whole)
            *reinterpret_cast<float2*>(p.part_ml + prow * 2) = make_float2(m, l);
          else if (p.lse)
            p.lse[orow] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : ninf();
        }
        tc_fence_before();
      }
      u += len;
      if (u >= u_end) break;
      attn_next<BN>(p, BM, &cur);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

template <bool BF16>
const void* attn_tc_fn(int dp);

}  // namespace sv
