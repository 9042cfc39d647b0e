// Attention of new tokens over a paged cache, tcgen05 kernel: pages that TMA can copy, heads of 64 to
// 128 values.
//
// One CTA per SM works through its run of (item, key tile) units, 128 keys a tile.  Eleven warps:
//   0-3, 4-7  softmax of half 0 and 1: a thread owns a row (TMEM lane): reads the row's 128 scores,
//             keeps the running maximum and sum, writes the probabilities back over the scores as
//             the second MMA's A operand, and rescales O in TMEM;
//   8         TMA producer: one box per page, head and 64 dims, 128-byte swizzle;
//   9         MMA issuer, one thread: S = Q K^T (both operands in shared memory) and O += P V (P in TMEM);
//   10        clears the value rows behind an item's last key (see below).
// TMEM (512 columns): S0 | S1 | O0 | O1, P_i in S_i's columns.  The two halves alternate: while one
// half's softmax runs, the tensor core works on the other's.  With more than 128 rows an item's halves
// are its rows 0-127 and 128-255, which share every key tile; with fewer they are the same rows over
// the even and the odd key tiles, joined at the end.  (One half alone would leave the tensor core, the
// softmax and the copies waiting for one another.)
//
// O is rescaled only when a row's maximum grows by more than 2^8 over the reference its exponentials
// use; until then the probabilities may reach 2^8, which neither type overflows and the final division
// by the sum undoes.  They are rounded to the operands' type (the A operand has B's): see the mma.sync kernel
// for what that costs.  S(j) is committed after the same half's previous P V in issue order, so a softmax
// thread that has seen S(j) may touch O.
//
// First tokens that stay visible behind a window (SINKS): the item's key tiles are those that hold them, then those of the
// window; what lies between is not looked at.  2 x 2048 tokens behind 14336, window 4096, 64 first tokens (279 GFLOP) 258 us:
// tiles that the mask cuts and an item's fixed cost every 35 tiles.
//
// Keys before the item's first one or at or beyond its last one: pages that lie wholly there are read at an
// out-of-range page coordinate, which TMA fills with zeros; the rest of the last page can hold anything, so its value
// rows are zeroed in shared memory before the MMA reads them (0 x NaN would be NaN); scores are
// selected, not multiplied.
//
// Bound and measured, heads of 128, bf16: 2 x 2048 tokens behind 14336, 32/8 heads (1.03 TFLOP) 667-745 us (by
// the machine and its power), 1.38-1.55 PFLOP/s, 73-82 % of the measured matrix rate: a half's softmax (1200 cycles a tile)
// and its two products (1024) follow one another, and the other half fills most of the gap.  32 x 17 tokens,
// 64/8 heads, ragged to 16384 keys (1.11 GB) 213-220 us, 5.0-5.2 TB/s, 74-76 % of the measured copy: 136 rows take two
// halves of 128.
//
// Over caches held in 4 bits (FP4) seven warps (8, 10 to 15) take the producer's place: they read codes and scales a tile
// ahead into registers, widen them to f16 (exactly: attention_fp4.cuh) and write them where the TMA boxes would lie; tokens
// that are not seen become zeros, so nothing has to be cleared, and any page size will do.  The queries of bf16 rows are
// f16 relative to a power of two at the row's largest value, the probabilities f16 up to 2^14.
//
// Measured, 4 bits: 32 x 17 tokens, 64/8 heads of 128, ragged to 16384 keys (352 MB, f16) 244 us; 2048 tokens behind 14336,
// 32/8 heads (515 GFLOP) 400 us, 1.29 PFLOP/s.  A key tile takes some 3300 cycles: a half's softmax 1850 (its latency: with
// 128 registers a thread 32 columns at a time), then its two products 1024 and the hand-overs.  The loaders are not in the
// way (without reads or without writes 241 to 258; 392 to 398), nor are the bytes (caches of 16 bits take 232 and 340-347
// us).  On the way, verify block and chunk: three loaders 557; 877, seven with page ids and codes ahead 357; 498,
// probabilities written 32 columns at a time so that 128 registers hold them 308; 471, one offset for keys and values 264;
// 447, maximum and exponentials in one pass 258; 406, whole heads and loose ones apart 246; 399, an item's fixed cost of
// five key tiles 242; 398, references as whole numbers 244; 400.  With whole heads of 128 bf16 spills 4 bytes of stores and
// 12 of loads a thread, f16 nothing.  Tried and dropped: copies into a ring of shared memory by a warp of its own 275; 433,
// loaders for keys and for values apart 313; 475, eleven loaders with 96 registers 268; 431, three with 168 310; 447,
// shares of a tile that take turns 243; 412, a quarter of the exponentials as polynomials 338; 583, 16 columns at a time
// 313; 539.
//
// Every wait is bounded: after `wait_limit` the kernel sets the status word, drains its copies and
// MMAs, frees TMEM and returns, its record for the combine kernel empty.
#pragma once

#include <cuda.h>

#include "attention_fp4.cuh"
#include "spec_async.cuh"

namespace sv {

constexpr int kTcThreads = 352;
constexpr int kTcLoaders = 7;        // warps that widen 4-bit keys and values
constexpr int kTcFp4Threads = 32 * (9 + kTcLoaders);
constexpr int kTcBN = 128;

// WIDE: row tiles of 256 (else 128), which take a second 128-row query buffer.
template <int DP, bool WIDE>
struct AttnTcGeom {
  static constexpr int kBM = WIDE ? 256 : 128;
  static constexpr int kTile = 128 * DP * 2;                 // 128 rows of Q, one tile's K or V
  static constexpr int kKStages = DP == 64 ? 5 : 3, kVStages = DP == 64 ? 5 : WIDE ? 2 : 3;
  static constexpr int kSmem = 1024 + (kBM / 128 + kKStages + kVStages) * kTile;
};

struct AttnTcBars {
  unsigned long long k_full[5], k_empty[5], v_full[5], v_empty[5];
  unsigned long long s_full[2], p_full[2], o_full[2], q_full[2];
  unsigned long long x_full, x_free;   // half 1's share of a joined item: there, and read
  unsigned long long clean_me[5], v_clean[5];   // a value slot to be cleared: asked for, done
  unsigned long long drain;
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
// Waits for this thread's TMEM loads; the registers pass through it, so that nothing reads them earlier.
__device__ __forceinline__ void tc_wait_ld(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// True in one lane of a converged warp, the same one every time.  (The compiler knows that a branch on
// it runs in one lane and keeps the operands of what is issued there in uniform registers.)
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// One arrival for the warp, after all its lanes.
__device__ __forceinline__ void mbar_arrive_warp(uint32_t bar) {
  __syncwarp();
  if (elected()) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
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
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
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
// 2^x of a whole number x <= 0 (or -inf), exactly.
__device__ __forceinline__ float tc_power(float x) {
  return x < -126.f ? 0.f : __uint_as_float(static_cast<uint32_t>(static_cast<int>(x) + 127) << 23);
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t f2_pack(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
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
  // Waits for the phase; false once the limit has passed or another warp gave up.  The clock (whose read
  // takes longer than most waits) is looked at only after a thousand polls.  (A number of polls that is no
  // constant makes a prompt chunk 3 % slower: 769 us for 748.)
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
#pragma unroll 1
    for (int k = 0; k < 1024; ++k)
      if (mbar_try(bar, parity)) return true;
    return slowly(bar, parity);
  }
  // The same for a whole warp.
  __device__ __forceinline__ bool warp(uint32_t bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, (*this)(bar, parity)) != 0;
  }
  __device__ __noinline__ bool slowly(uint32_t bar, uint32_t parity) const {
    const unsigned long long t0 = global_ns();
    while (true) {
#pragma unroll 1
      for (int k = 0; k < 256; ++k)
        if (mbar_try(bar, parity)) return true;
      if (*abort) return false;
      if (static_cast<long long>(global_ns() - t0) > limit) return give_up();
    }
  }
  __device__ __forceinline__ bool give_up() const {
    *abort = 1;
    atomicOr(status, kStatusTimeout);
    return false;
  }
};

// A loader's share of a tile's keys (or values) in registers: units of 32 values, 16 bytes of codes and two scales.
template <int DP>
struct TcFp4Share {
  static constexpr int kLanes = DP / 32;             // lanes of a key
  static constexpr int kKeys = 32 / kLanes;          // keys of a step
  static constexpr int kSteps = kTcBN / kKeys, kMine = (kSteps + kTcLoaders - 1) / kTcLoaders;
  static constexpr int kRounds = (kMine * kKeys + 31) / 32;   // keys of a loader's share, 32 at a time
  static_assert(32 % kKeys == 0, "a step's keys are held by consecutive lanes");
  static constexpr uint32_t kNone = 0xffffffffu;
  uint4 codes[kMine];
  uint16_t scales[kMine];
  // This lane's key of its step i (at or beyond the tile's end: none).  Lanes 0 to 7 have 8 keys (16 where a key is two
  // lanes' work) and the same place in them, so that a store phase falls on distinct banks.
  static __device__ __forceinline__ int key(int loader, int i, int lane) { return (i * kTcLoaders + loader) * kKeys + lane % kKeys; }
  // Reads this lane's units of the keys at the given scales (offset in bytes; none: zeros).  The codes lie 8 times as far
  // from their base, and the bases are those of the lane's place in a key.
  template <bool WHOLE>
  __device__ __forceinline__ void load(const uint8_t* codes_at, const uint8_t* scales_at, const uint32_t (&at)[kMine], int D,
                                       int lane) {
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const uint8_t* x = codes_at + static_cast<unsigned long long>(at[i]) * 8;
      const uint8_t* y = scales_at + at[i];
      if (WHOLE) {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0xffffffff;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t"
            "mov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\tmov.b16 %4, 0;\n\t"
            "@p ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%6];\n\t@p ld.global.nc.b16 %4, [%7];\n\t}"
            : "=&r"(codes[i].x), "=&r"(codes[i].y), "=&r"(codes[i].z), "=&r"(codes[i].w), "=&h"(scales[i])
            : "r"(at[i]), "l"(x), "l"(y));
      } else {
        const int c = lane / kKeys;
        codes[i] = make_uint4(0, 0, 0, 0);
        scales[i] = 0;
        if (at[i] == kNone || c * 32 >= D) continue;
        const uint2 a = __ldg(reinterpret_cast<const uint2*>(x));
        codes[i].x = a.x;
        codes[i].y = a.y;
        scales[i] = __ldg(y);
        if (c * 32 + 16 < D) {
          const uint2 b = __ldg(reinterpret_cast<const uint2*>(x) + 1);
          codes[i].z = b.x;
          codes[i].w = b.y;
          scales[i] = static_cast<uint16_t>(scales[i] | __ldg(y + 1) << 8);
        }
      }
    }
  }
  // Writes them as f16 into a tile: 64-value blocks of 128 rows of 128 bytes, 16-byte pieces permuted by the row.
  __device__ __forceinline__ void store(uint32_t tile, int loader, int lane) const {
    const int c = lane / kKeys;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int r = key(loader, i, lane);
      if (i * kTcLoaders + loader >= kSteps) break;   // the same for the whole warp
      const uint32_t two = fp4_scales(scales[i]), f0 = __byte_perm(two, two, 0x1010), f1 = __byte_perm(two, two, 0x3232);
      const uint32_t at = tile + (c / 2) * 16384 + r * 128 + ((((c & 1) * 4) ^ (r & 7)) << 4);
      const uint32_t w[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t f = k < 2 ? f0 : f1;
        uint32_t v[4];
        fp4_pairs(w[k], v);
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at ^ (k << 4)), "r"(mul2(v[0], f)), "r"(mul2(v[1], f)),
                     "r"(mul2(v[2], f)), "r"(mul2(v[3], f))
                     : "memory");
      }
    }
  }
};

// WHOLE (FP4): heads of DP values, codes and scales aligned to whole pieces.  (As a branch of the loop: 5 % slower.)
template <bool BF16, int DP, bool WIDE, bool SINKS, bool FP4, bool WHOLE>
__global__ void __launch_bounds__(FP4 ? kTcFp4Threads : kTcThreads, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const AttnParams p) {
  using A = AttnType<BF16>;
  using M = AttnType<BF16 && !FP4>;   // the products' operands
  constexpr int THREADS = FP4 ? kTcFp4Threads : kTcThreads;
  constexpr float kShift = FP4 ? kFp4Shift : 0.f;   // of the probabilities, in powers of two
  using Geo = AttnTcGeom<DP, WIDE>;
  constexpr int BM = Geo::kBM, BN = kTcBN, SUB = DP / 64, KST = Geo::kKStages, VST = Geo::kVStages, TILE = Geo::kTile;
  extern __shared__ uint8_t smem_raw[];
  __shared__ AttnSchedSmem<THREADS> sched;
  __shared__ __align__(8) AttnTcBars bars;
  __shared__ float2 s_ml[128];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t s_q = base, s_k = base + (BM / 128) * TILE, s_v = s_k + KST * TILE;

  const AttnSplit split = attn_split<BN, SINKS>(p, BM, sched);
  const int cta = blockIdx.x;
  asm volatile("griddepcontrol.launch_dependents;");
  if (cta >= split.n) {
    if (tid == 0) attn_leave_join(p, split, cta, BM, nullptr, false);
    return;
  }
  const long long u_begin = split.begin(cta), u_end = split.begin(cta + 1);
  AttnCursor cur = attn_locate<BN, SINKS>(p, BM, u_begin, sched);
  int k0, k1;   // the item's key tiles that are this CTA's
  cur.share(p, u_begin, u_end, &k0, &k1);
  if (k1 <= k0) {   // nothing but an item's overhead
    if (tid == 0) attn_leave_join(p, split, cta, BM, nullptr, false);
    return;
  }

  if (tid == 0) {
    // A CTA that gives up leaves this empty record: the combine kernel runs all the same, and what the
    // workspace held before must not lead it anywhere.
    attn_leave_join(p, split, cta, BM, nullptr, false);
    s_abort = 0;
    for (int i = 0; i < 5; ++i) {
      mbar_init(smem_addr(&bars.k_full[i]), FP4 ? kTcLoaders : 1);
      mbar_init(smem_addr(&bars.k_empty[i]), 1);
      mbar_init(smem_addr(&bars.v_full[i]), FP4 ? kTcLoaders : 1);
      mbar_init(smem_addr(&bars.v_empty[i]), 1);
      mbar_init(smem_addr(&bars.clean_me[i]), 1);
      mbar_init(smem_addr(&bars.v_clean[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&bars.s_full[i]), 1);
      mbar_init(smem_addr(&bars.p_full[i]), 4);
      mbar_init(smem_addr(&bars.o_full[i]), 1);
      mbar_init(smem_addr(&bars.q_full[i]), 4);
    }
    mbar_init(smem_addr(&bars.x_full), 4);
    mbar_init(smem_addr(&bars.x_free), 4);
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
  unsigned issued = 0;   // producer: key tiles whose copies were issued

  if (FP4 && warp >= 8 && warp != 9) {
    // ------------------------------------------------------------------ loaders of 4-bit keys and values
    // In the order in which the issuer asks: keys of tile g + 1, values of tile g.  Both were read a tile before, and the
    // page ids for that a tile before that, so no latency of the table or of memory stands between two tiles.
    using Share = TcFp4Share<DP>;
    const int loader = warp == 8 ? 0 : warp - 9, P = p.c.page_size;
    struct Fetched {   // of a tile's keys: lane n has the page and slot of key n of the warp's share (slot -1: none)
      int pg[Share::kRounds], in[Share::kRounds], head;
      bool there;      // there is such a tile
    };
    struct Places {    // offsets of this lane's keys (Share::load)
      uint32_t at[Share::kMine];
      bool there;
    };
    int lo, hi, j = 0;   // the item's keys; its tile that is fetched next
    const int32_t* table;
    auto begin_item = [&] {
      const int r0 = cur.t * BM, r1 = min(cur.req.nq * p.G, r0 + BM);
      attn_keys(p, cur.req, r0, r1, &lo, &hi);
      table = p.c.table + static_cast<long long>(cur.b) * p.c.table_stride;
    };
    begin_item();
    bool left = true;    // a tile is left to fetch
    auto fetch = [&](Fetched& x) {
      x.there = left;
      if (!left) return;
      const int key0 = cur.template tile<SINKS>(k0 + j) * BN;
      x.head = cur.h;
#pragma unroll
      for (int n = 0; n < Share::kRounds; ++n) {
        const int at = n * 32 + lane;
        const int r = (at / Share::kKeys * kTcLoaders + loader) * Share::kKeys + at % Share::kKeys, key = key0 + r;
        x.pg[n] = -1;
        x.in[n] = -1;
        if (r < BN && key < hi && (key >= lo || (SINKS && key < p.sinks))) {
          // key / P: the product with floor(2^32 / P) is the quotient or one less
          int col = static_cast<int>(__umulhi(static_cast<unsigned>(key), p.page_inv));
          int in = key - col * P;
          if (in >= P) {
            ++col;
            in -= P;
          }
          x.in[n] = in;
          x.pg[n] = __ldg(table + col);
        }
      }
      if (++j < k1 - k0) return;
      left = attn_next<BN, SINKS>(p, BM, u_end, &cur);
      if (!left) return;
      cur.share(p, u_begin, u_end, &k0, &k1);
      begin_item();
      j = 0;
    };
    // Page ids outside the cache are reported and read as zeros.  Offsets of scales are 32-bit numbers (the host sees to it).
    auto place = [&](const Fetched& x, Places& to) {
      to.there = x.there;
      uint32_t at[Share::kRounds];
#pragma unroll
      for (int n = 0; n < Share::kRounds; ++n) {
        const bool bad = x.pg[n] < 0 || x.pg[n] >= p.c.pages;
        if (bad && x.in[n] >= 0) atomicOr(p.status, kStatusPageRange);
        at[n] = bad ? Share::kNone
                    : static_cast<uint32_t>(x.pg[n]) * static_cast<uint32_t>(p.s.k_page) +
                          static_cast<uint32_t>(x.in[n]) * static_cast<uint32_t>(p.s.k_token) +
                          static_cast<uint32_t>(x.head) * static_cast<uint32_t>(p.s.k_head);
      }
#pragma unroll
      for (int i = 0; i < Share::kMine; ++i)
        to.at[i] = __shfl_sync(0xffffffffu, at[i * Share::kKeys / 32], (i * Share::kKeys + lane % Share::kKeys) % 32);
    };
    Share k, v;
    const int in_key = lane / Share::kKeys;   // this lane's 32 values of a key
    const uint8_t *k_codes = p.c.k + in_key * 16, *v_codes = p.c.v + in_key * 16;
    const uint8_t *k_scales = p.s.k + in_key * 2, *v_scales = p.s.v + in_key * 2;
    auto load_k = [&](const Places& x) { k.template load<WHOLE>(k_codes, k_scales, x.at, p.c.D, lane); };
    auto load_v = [&](const Places& x) { v.template load<WHOLE>(v_codes, v_scales, x.at, p.c.D, lane); };
    bool ok = p.wait_limit > 0 || wait.give_up();
    unsigned g = 0;   // key tiles of this CTA so far
    auto put_k = [&](unsigned n) -> bool {
      const unsigned st = n % KST;
      if (!wait.warp(smem_addr(&bars.k_empty[st]), (n / KST & 1) ^ 1)) return false;
      k.store(s_k + st * TILE, loader, lane);
      fence_async_smem();
      mbar_arrive_warp(smem_addr(&bars.k_full[st]));
      return true;
    };
    auto put_v = [&](unsigned n) -> bool {
      const unsigned st = n % VST;
      if (!wait.warp(smem_addr(&bars.v_empty[st]), (n / VST & 1) ^ 1)) return false;
      v.store(s_v + st * TILE, loader, lane);
      fence_async_smem();
      mbar_arrive_warp(smem_addr(&bars.v_full[st]));
      return true;
    };
    Fetched fetched;
    Places next, after;   // tiles g + 1, g + 2
    fetch(fetched);
    place(fetched, next);
    load_k(next);
    load_v(next);
    fetch(fetched);
    ok = ok && put_k(0);
    place(fetched, next);
    if (next.there) load_k(next);
    fetch(fetched);
    while (ok) {
      place(fetched, after);
      if (next.there) {
        if (!(ok = put_k(g + 1))) break;
        if (after.there) load_k(after);
      }
      if (!(ok = put_v(g)) || !next.there) break;
      load_v(next);
      fetch(fetched);
      next = after;
      ++g;
    }
  } else if (!FP4 && warp == 8) {
    // ------------------------------------------------------------------------------ TMA producer
    const int P = p.c.page_size, rows = min(P, BN), boxes = BN / rows;   // boxes of 64 dims per tile
    unsigned g = 0;                                                      // key tiles of this CTA so far
    // without a limit the first wait gives up at once; the other warps, whose tiles never come, follow
    bool ok = p.wait_limit > 0 || wait.give_up();
    while (ok) {
      const int len = k1 - k0;
      const int r0 = cur.t * BM, r1 = min(cur.req.nq * p.G, r0 + BM);
      int lo, hi;
      attn_keys(p, cur.req, r0, r1, &lo, &hi);
      const int32_t* table = p.c.table + static_cast<long long>(cur.b) * p.c.table_stride;
      for (int j = 0; ok && j < len; ++j, ++g) {
        // this lane's boxes: page `i` of the tile (i = lane: at most 16 pages of 8 tokens and more)
        const int kt = cur.template tile<SINKS>(k0 + j), key = kt * BN + lane * rows;
        int pg = p.c.pages;   // out of range: zeros.  So too what lies wholly before the window: its page may be gone
        if (lane < boxes && key < hi && (key + rows > lo || (SINKS && key < p.sinks))) {
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
          ok = wait.warp(empty, ph ^ 1);
          if (!ok) break;
          if (elected()) mbar_arrive_tx(full, TILE);
          __syncwarp();
          if (lane < boxes) {
            const uint32_t dst = (which ? s_v : s_k) + st * TILE + lane * rows * 128;
#pragma unroll
            for (int s = 0; s < SUB; ++s) tma_box(dst + s * 128 * 128, which ? &map_v : &map_k, s * 64, tok, cur.h, pg, full);
          }
          __syncwarp();
          if (which && (kt + 1) * BN > hi) mbar_arrive_warp(smem_addr(&bars.clean_me[st]));
        }
      }
      if (!attn_next<BN, SINKS>(p, BM, u_end, &cur)) break;
      cur.share(p, u_begin, u_end, &k0, &k1);
    }
    issued = g;
  } else if (warp == 9) {
    // -------------------------------------------------------------------------------- MMA issuer
    // The whole loop runs in one elected thread: a warp-wide wait costs three times a thread's, and
    // whatever the issuer spends between two products is time the tensor core stands still.
    constexpr uint32_t kType = BF16 && !FP4 ? 1u : 0u;
    constexpr uint32_t kCommon = (1u << 4) | (kType << 7) | (kType << 10) | ((128u >> 4) << 24);
    constexpr uint32_t kIdescS = kCommon | ((128u >> 3) << 17);
    constexpr uint32_t kIdescO = kCommon | (1u << 16) | ((static_cast<uint32_t>(DP) >> 3) << 17);
    bool ok = true;
    if (elected()) {
      // rings of slots: the next one to use, its phase, the operand's descriptor
      struct Ring {
        uint32_t slot, phase, full, empty;
        uint64_t desc;
      };
      const uint64_t desc_q = tc_desc(s_q, 16), desc_k = tc_desc(s_k, 16), desc_v = tc_desc(s_v, 16384);
      Ring kr = {0, 0, smem_addr(bars.k_full), smem_addr(bars.k_empty), desc_k};
      Ring vr = {0, 0, smem_addr(bars.v_full), smem_addr(bars.v_empty), desc_v};
      auto next_k = [&] {
        kr.full += 8;
        kr.empty += 8;
        kr.desc += TILE >> 4;
        if (++kr.slot == KST) kr = {0, kr.phase ^ 1, smem_addr(bars.k_full), smem_addr(bars.k_empty), desc_k};
      };
      auto next_v = [&] {
        vr.full += 8;
        vr.empty += 8;
        vr.desc += TILE >> 4;
        if (++vr.slot == VST) vr = {0, vr.phase ^ 1, smem_addr(bars.v_full), smem_addr(bars.v_empty), desc_v};
      };
      unsigned pv_phase = 0, q_phase = 0, cleaned = 0;   // phases, a bit per half or slot
      const uint32_t bar_s = smem_addr(bars.s_full), bar_o = smem_addr(bars.o_full);
      const uint32_t bar_p = smem_addr(bars.p_full);
      auto issue_s = [&](int half, uint64_t q) {
        const uint32_t d = tmem + half * 128;
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          const uint32_t off = ((k / 4) * 16384 + (k % 4) * 32) >> 4;
          tc_mma_ss(d, q + off, kr.desc + off, kIdescS, k > 0);
        }
        tc_commit(bar_s + half * 8);
      };
      // O += P V of one half
      auto add_pv = [&](int half, bool acc) -> bool {
        const uint32_t a = tmem + half * 128, d = a + 256;
        if (!wait(bar_p + half * 8, pv_phase >> half & 1)) return false;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 8; ++k) tc_mma_ts(d, a + k * 8, vr.desc + (k * 2048 >> 4), kIdescO, acc || k > 0);
        pv_phase ^= 1u << half;
        return true;
      };
      while (ok) {
        const int len = k1 - k0;
        const int r0 = cur.t * BM, r1 = min(cur.req.nq * p.G, r0 + BM);
        const bool joined = r1 - r0 <= 128;
        int lo, hi;
        attn_keys(p, cur.req, r0, r1, &lo, &hi);
        const int clean_from = cur.template number<SINKS>(hi / BN) - k0;   // tiles from here on end behind the item's last key
        for (int h = 0; ok && h < (joined ? 1 : 2); ++h) {
          ok = wait(smem_addr(&bars.q_full[h]), q_phase >> h & 1);
          q_phase ^= 1u << h;
        }
        // the first scores of both halves
        for (int j = 0; ok && j < (joined ? min(len, 2) : 1); ++j) {
          ok = wait(kr.full, kr.phase);
          if (!ok) break;
          tc_fence_after();
          issue_s(joined ? j : 0, desc_q);
          if (!joined) issue_s(1, desc_q + (TILE >> 4));
          tc_commit(kr.empty);
          next_k();
        }
        for (int j = 0; ok && j < len; ++j) {
          ok = wait(vr.full, vr.phase);
          if (!FP4 && ok && j >= clean_from) {
            ok = wait(smem_addr(&bars.v_clean[vr.slot]), cleaned >> vr.slot & 1);
            cleaned ^= 1u << vr.slot;
          }
          if (!ok) break;
          const int first = joined ? j & 1 : 0;
          const bool more = j + (joined ? 2 : 1) < len;   // the half has a key tile after this one
          if (!(ok = add_pv(first, j >= (joined ? 2 : 1)))) break;
          if (more) {
            if (!(ok = wait(kr.full, kr.phase))) break;
            tc_fence_after();
            issue_s(first, desc_q);
          } else {
            tc_commit(bar_o + first * 8);
          }
          if (!joined) {
            if (!(ok = add_pv(1, j > 0))) break;
            if (more)
              issue_s(1, desc_q + (TILE >> 4));
            else
              tc_commit(bar_o + 8);
          }
          tc_commit(vr.empty);
          next_v();
          if (more) {
            tc_commit(kr.empty);
            next_k();
          }
        }
        if (!ok || !attn_next<BN, SINKS>(p, BM, u_end, &cur)) break;
        cur.share(p, u_begin, u_end, &k0, &k1);
      }
      if (!ok) {   // gave up: the MMAs in flight finish before TMEM is freed
        tc_commit(smem_addr(&bars.drain));
        const unsigned long long t0 = global_ns();
        while (!mbar_try(smem_addr(&bars.drain), 0) && global_ns() - t0 < 100000000ull) {
        }
      }
    }
    __syncwarp();
  } else if (!FP4 && warp == 10) {
    // ---------------------------------------------------------------- value rows behind the last key
    // The producer asks for a slot after it has armed the slot's v_full; the slot is not armed again
    // before the issuer has seen it cleared, so no phase of the three barriers is ever missed.
    unsigned g = 0, asked = 0;   // phases of clean_me, a bit per slot
    bool ok = true;
    while (ok) {
      const int len = k1 - k0;
      const int r0 = cur.t * BM, r1 = min(cur.req.nq * p.G, r0 + BM);
      int lo, hi;
      attn_keys(p, cur.req, r0, r1, &lo, &hi);
      for (int j = max(cur.template number<SINKS>(hi / BN) - k0, 0); ok && j < len; ++j) {
        const unsigned t = g + j, st = t % VST;
        ok = wait.warp(smem_addr(&bars.clean_me[st]), asked >> st & 1);
        asked ^= 1u << st;
        if (ok) ok = wait.warp(smem_addr(&bars.v_full[st]), (t / VST) & 1);
        if (!ok) break;
        const int valid = max(hi - cur.template tile<SINKS>(k0 + j) * BN, 0);
        for (int i = valid * 8 + lane; i < BN * 8; i += 32)
#pragma unroll
          for (int s = 0; s < SUB; ++s)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(s_v + st * TILE + s * 16384 + i * 16), "r"(0u) : "memory");
        fence_async_smem();
        mbar_arrive_warp(smem_addr(&bars.v_clean[st]));
      }
      g += len;
      if (!attn_next<BN, SINKS>(p, BM, u_end, &cur)) break;
      cur.share(p, u_begin, u_end, &k0, &k1);
    }
  } else {
    // ------------------------------------------------------------------------------------ softmax
    const int half = warp >> 2, row = tid & 127;   // row of the half = TMEM lane
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + half * 128, t_o = tmem + lanes + 256 + half * 128;
    const uint32_t bar_s = smem_addr(&bars.s_full[half]);
    unsigned tiles = 0, segs = 0, joins = 0;
    bool later = false;             // not the CTA's first item
    bool ok = true, owed = false;   // owed: half 0 may still read this half's O and statistics
    // Writes this half's queries of an item where the MMAs read them.  Returns the factor of the scores.
    auto load_q = [&](const AttnCursor& it) -> float {
      const int r0 = it.t * BM, r1 = min(it.req.nq * p.G, r0 + BM);
      const bool joined = r1 - r0 <= 128;
      const int r = r0 + (joined ? 0 : half * 128) + row;
      const bool mine = r < r1;
      const int tok = it.req.q0 + attn_token(p, r), head = it.h * p.G + r - (attn_token(p, r)) * p.G;
      const uint8_t* src = p.q + (tok * p.q_token + head * p.q_head) * 2;
      float scale_log2 = p.scale_log2, down = 1.f;
      if constexpr (FP4) {
        // the row in f16; both halves need its power of two, the one that owns it writes it
        if (BF16) {
          float top = 0.f;
#pragma unroll
          for (int c = 0; c < DP / 8; ++c) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (mine && c * 8 < p.c.D) v = __ldg(reinterpret_cast<const uint4*>(src + c * 16));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xffff0000u))));
          }
          scale_log2 *= fp4_query_power(top, &down);
        }
        scale_log2 = fmaxf(scale_log2, kFp4Least);
      }
      if (half == 0 || !joined) {
        const uint32_t dst = s_q + half * TILE + row * 128;
#pragma unroll
        for (int c = 0; c < DP / 8; ++c) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (mine && c * 8 < p.c.D) v = __ldg(reinterpret_cast<const uint4*>(src + c * 16));
          uint32_t w[4] = {v.x, v.y, v.z, v.w};
          if (FP4 && BF16) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = M::pack(__uint_as_float(w[e] << 16) * down, __uint_as_float(w[e] & 0xffff0000u) * down);
          }
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst + (c / 8) * 16384 + (((c & 7) ^ (row & 7)) << 4)),
                       "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                       : "memory");
        }
        fence_async_smem();
        mbar_arrive_warp(smem_addr(&bars.q_full[half]));
      }
      return scale_log2;
    };
    float scale_log2 = p.scale_log2;
    if (!FP4) load_q(cur);
    while (ok) {
      const int len = k1 - k0;
      const int r0 = cur.t * BM, r1 = min(cur.req.nq * p.G, r0 + BM);
      const bool joined = r1 - r0 <= 128;
      const int h0 = r0 + (joined ? 0 : half * 128), r = h0 + row;
      const bool mine = r < r1;
      const bool busy = h0 + (warp & 3) * 32 < r1;   // some row of this warp exists
      if (FP4) scale_log2 = load_q(cur);
      if (owed) {
        ok = wait.warp(smem_addr(&bars.x_free), (joins - 1) & 1);
        if (!ok) break;
        tc_fence_after();
        owed = false;
      }
      int row_lo = 0, row_hi = 0;
      if (mine) attn_keys(p, cur.req, r, r + 1, &row_lo, &row_hi);
      // key tiles inside [w_lo, w_hi) need no mask for any row of the warp
      const int w_hi = __reduce_min_sync(0xffffffffu, mine ? row_hi : 0x7fffffff);
      const int w_lo = __reduce_max_sync(0xffffffffu, mine ? row_lo : 0);
      const int j0 = joined ? half : 0, step = joined ? 2 : 1;
      float m = ninf(), l = 0.f;
      for (int j = j0; j < len; j += step, ++tiles) {
        ok = wait.warp(bar_s, tiles & 1);
        if (!ok) break;
        tc_fence_after();
        if (FP4 && busy) {
          // The same with 128 registers a thread: the probabilities of 32 columns are written before the next are worked
          // on (over scores that have been read).  An item's first reference comes from a pass over all columns; where 32
          // columns outgrow it, they are read again, and what was written against the old one is rescaled.  References are
          // whole numbers (the maximum rounded up), so that the factor is a power of two: f16 probabilities, the sum and O
          // are rescaled exactly.
          const int key0 = cur.template tile<SINKS>(k0 + j) * BN, lo = row_lo - key0, hi = row_hi - key0;
          const int sinks = SINKS ? p.sinks - key0 : 0;
          const bool masked = key0 + BN > w_hi || key0 < w_lo;
          const uint64_t scale2 = f2_pack(scale_log2, scale_log2);
          auto mask = [&](uint32_t (&s)[32], int c) {
            if (masked) {
#pragma unroll
              for (int i = 0; i < 32; ++i) s[i] = (c + i >= lo || (SINKS && c + i < sinks)) && c + i < hi ? s[i] : 0xff800000u;
            }
          };
          if (__any_sync(0xffffffffu, mine && m == ninf())) {
            float t[4] = {ninf(), ninf(), ninf(), ninf()};
#pragma unroll 1
            for (int c = 0; c < BN; c += 32) {
              uint32_t s[32];
              tc_ld32(t_s + c, s);
              tc_wait_ld(s);
              mask(s, c);
#pragma unroll
              for (int i = 0; i < 16; ++i)
                t[i & 3] = fmaxf(fmaxf(t[i & 3], __uint_as_float(s[2 * i])), __uint_as_float(s[2 * i + 1]));
            }
            if (m == ninf()) m = ceilf(fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * scale_log2);   // O and the sum are zero so far
          }
          // 32 columns: exponentials against the reference, their sum, the maximum (scaled: the scale is positive)
          auto work = [&](uint32_t (&s)[32], int c) {
            uint32_t pk[16];
            float sums, top;
            auto pass = [&] {
              const float ref = (m == ninf() ? 0.f : m) - kShift;
              const uint64_t ref2 = f2_pack(-ref, -ref);
              uint64_t sum[2] = {0ull, 0ull};
              float t[4] = {ninf(), ninf(), ninf(), ninf()};
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float x0 = __uint_as_float(s[2 * i]), x1 = __uint_as_float(s[2 * i + 1]);
                t[i & 3] = fmaxf(fmaxf(t[i & 3], x0), x1);
                float e0, e1;
                f2_unpack(f2_fma(f2_pack(x0, x1), scale2, ref2), e0, e1);
                e0 = ex2(e0);
                e1 = ex2(e1);
                sum[i & 1] = f2_add(sum[i & 1], f2_pack(e0, e1));
                pk[i] = M::pack(e0, e1);
              }
              float a, b;
              f2_unpack(f2_add(sum[0], sum[1]), a, b);
              sums = a + b;
              top = fmaxf(m, fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * scale_log2);
            };
            mask(s, c);
            pass();
            if (__any_sync(0xffffffffu, top - m > kFp4Grow)) {
              top = ceilf(top);
              const float f = tc_power(m - (top == ninf() ? 0.f : top));
              l *= f;
              m = top;
              if (j > j0) {
#pragma unroll 1
                for (int d = 0; d < DP; d += 32) {
                  tc_ld32(t_o + d, s);
                  tc_wait_ld(s);
#pragma unroll
                  for (int i = 0; i < 32; ++i) s[i] = __float_as_uint(__uint_as_float(s[i]) * f);
                  tc_st32(t_o + d, s);
                }
              }
              tc_wait_st();
#pragma unroll 1
              for (int d = 0; d < c / 2; d += 16) {   // 16 columns hold 32 probabilities (the 16 behind them are read along)
                tc_ld32(t_s + d, s);
                tc_wait_ld(s);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&s[i]));
                  s[i] = M::pack(y.x * f, y.y * f);
                }
                tc_st16(t_s + d, s);
              }
              tc_wait_st();
              tc_ld32(t_s + c, s);
              tc_wait_ld(s);
              mask(s, c);
              pass();
            }
            l += sums;
            tc_st16(t_s + c / 2, pk);
          };
#pragma unroll 1
          for (int c = 0; c < BN; c += 32) {
            uint32_t s[32];
            tc_ld32(t_s + c, s);
            tc_wait_ld(s);
            work(s, c);
          }
          tc_wait_st();
        }
        if (!FP4 && busy) {
          // One pass over the scores, 32 columns at a time with the next ones in flight: maximum,
          // exponentials against the reference so far, their sum.  Only where the maximum has outgrown
          // the reference (always in an item's first tile) the pass is done again with the new one.
          const int key0 = cur.template tile<SINKS>(k0 + j) * BN, lo = row_lo - key0, hi = row_hi - key0;
          const int sinks = SINKS ? p.sinks - key0 : 0;
          const bool masked = key0 + BN > w_hi || key0 < w_lo;
          const uint64_t scale2 = f2_pack(scale_log2, scale_log2);
          uint32_t pk[64];
          while (true) {
            const float ref = m == ninf() ? 0.f : m;
            const uint64_t ref2 = f2_pack(-ref, -ref);
            uint32_t s[2][32];
            float t[4] = {ninf(), ninf(), ninf(), ninf()};
            uint64_t sum[2] = {0ull, 0ull};
            tc_ld32(t_s, s[0]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t (&x)[32] = s[c & 1];
              tc_wait_ld(x);
              if (c < 3) tc_ld32(t_s + (c + 1) * 32, s[(c + 1) & 1]);
              if (masked) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  x[i] = (c * 32 + i >= lo || (SINKS && c * 32 + i < sinks)) && c * 32 + i < hi ? x[i] : 0xff800000u;
              }
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float x0 = __uint_as_float(x[2 * i]), x1 = __uint_as_float(x[2 * i + 1]);
                t[i & 3] = fmaxf(fmaxf(t[i & 3], x0), x1);
                float e0, e1;
                f2_unpack(f2_fma(f2_pack(x0, x1), scale2, ref2), e0, e1);
                e0 = ex2(e0);
                e1 = ex2(e1);
                sum[i & 1] = f2_add(sum[i & 1], f2_pack(e0, e1));
                pk[c * 16 + i] = M::pack(e0, e1);
              }
            }
            // in units of the scaled scores (the scale is positive)
            const float top = fmaxf(m, fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * scale_log2);
            const bool grow = top - m > 8.f || (m == ninf() && top > m);
            if (!__any_sync(0xffffffffu, grow)) {
              float a, b, c, d;
              f2_unpack(sum[0], a, b);
              f2_unpack(sum[1], c, d);
              l += (a + b) + (c + d);
              break;
            }
            const float f = ex2(m - (top == ninf() ? 0.f : top));
            l *= f;
            m = top;
            if (j > j0) {
#pragma unroll 1
              for (int c = 0; c < DP / 32; ++c) {
                tc_ld32(t_o + c * 32, s[0]);
                tc_wait_ld(s[0]);
#pragma unroll
                for (int i = 0; i < 32; ++i) s[0][i] = __float_as_uint(__uint_as_float(s[0][i]) * f);
                tc_st32(t_o + c * 32, s[0]);
              }
            }
          }
          tc_st32(t_s, pk);
          tc_st32(t_s + 32, pk + 32);
          tc_wait_st();
        }
        tc_fence_before();
        mbar_arrive_warp(smem_addr(&bars.p_full[half]));
      }
      if (!ok) break;
      // The next item's queries, before this one's rows are written: its first scores are on their way meanwhile (2 x 2048
      // tokens behind 14336 745 -> 734 us, 64 prompts of 300 behind 300 298 -> 264; over 4 bits 1 % slower).  The MMAs that read
      // the old ones are done: the half's own when its last scores are there; of a joined item's two halves, which share
      // them, when half 0's O is (it comes after both halves' last scores).
      auto wait_o = [&] {
        if (j0 < len) {
          ok = wait.warp(smem_addr(&bars.o_full[half]), segs & 1);
          ++segs;
        }
      };
      AttnCursor next = cur;
      bool more = false;
      if constexpr (!FP4) {
        more = attn_next<BN, SINKS>(p, BM, u_end, &next);
        if (joined) wait_o();
        if (!ok) break;
        if (more) load_q(next);
        if (!joined) wait_o();
      } else {
        wait_o();
      }
      if (!ok) break;
      if (j0 < len) tc_fence_after();
      float f0 = 1.f, f1 = 0.f;   // the halves' factors
      if (joined) {
        ++joins;
        if (half == 1) {
          s_ml[row] = make_float2(m, l);
          tc_fence_before();
          mbar_arrive_warp(smem_addr(&bars.x_full));
          owed = true;
        } else {
          ok = wait.warp(smem_addr(&bars.x_full), (joins - 1) & 1);
          if (!ok) break;
          tc_fence_after();
          const float2 other = s_ml[row];
          const float top = fmaxf(m, other.x), ref = top == ninf() ? 0.f : top;
          f0 = ex2(m - ref);
          f1 = ex2(other.x - ref);
          m = top;
          l = l * f0 + other.y * f1;
        }
      }
      if (half == 0 || !joined) {
        const bool whole = len == cur.count;
        const float inv = whole ? attn_factor(l, FP4 ? p.v_unit : 1.f) : 1.f;
        f0 *= inv;
        f1 *= inv;
        const bool both = joined && len > 1;
        const int tok = attn_token(p, r);
        const long long orow = static_cast<long long>(cur.req.q0 + tok) * p.Hq + cur.h * p.G + (r - tok * p.G);
        const long long prow = static_cast<long long>(2 * cta + (later ? 1 : 0)) * BM + (r - r0);
        if (busy) {
#pragma unroll 1
          for (int c = 0; c < DP / 32; ++c) {
            uint32_t o[32], o1[32];
            __syncwarp();
            tc_ld32(t_o + c * 32, o);
            tc_ld32(t_o + (both ? 128 : 0) + c * 32, o1);
            tc_wait_ld(o);
            tc_wait_ld(o1);
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              const int d = c * 32 + i;
              if (!mine || d >= p.c.D) continue;
              float f[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                f[e] = __uint_as_float(o[i + e]) * f0;
                if (both) f[e] = fmaf(__uint_as_float(o1[i + e]), f1, f[e]);
              }
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
            *reinterpret_cast<float2*>(p.part_ml + prow * 2) = make_float2(m - kShift, l);
          else if (p.lse)
            p.lse[orow] = attn_lse(m - kShift, l);
        }
        tc_fence_before();
        if (joined) mbar_arrive_warp(smem_addr(&bars.x_free));
      }
      if constexpr (FP4) {
        next = cur;
        more = attn_next<BN, SINKS>(p, BM, u_end, &next);
      }
      if (!more) {
        if (tid == 0) attn_leave_join(p, split, cta, BM, &cur, later);
        break;
      }
      cur = next;
      cur.share(p, u_begin, u_end, &k0, &k1);
      later = true;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (!FP4 && warp == 8 && s_abort) {   // gave up: the copies in flight still land before the block's memory is given back
    for (unsigned i = issued > KST + VST ? issued - KST - VST : 0; i <= issued; ++i) {
      const unsigned long long t0 = global_ns();
      while (!(mbar_try(smem_addr(&bars.k_full[i % KST]), (i / KST) & 1) && mbar_try(smem_addr(&bars.v_full[i % VST]), (i / VST) & 1)) &&
             global_ns() - t0 < 20000000ull) {
      }
    }
  }
  if (warp == 9) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

template <bool BF16, bool SINKS>
const void* attn_tc_fn(int dp, bool wide);
template <bool BF16>
const void* attn_tc_fp4_fn(int dp, bool wide, bool whole);

}  // namespace sv
