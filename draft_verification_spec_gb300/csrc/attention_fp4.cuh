// Attention of new tokens over a paged cache held in 4 bits (step_internal.h: Fp4Scales), mma.sync kernel: any page
// size, head sizes up to 256, tiles of 8, 16 or 32 rows.
//
// The same formula and the same work division as the kernel over 16-bit caches (attention_mma.cuh), over
//   k = unit scale[block] code: code e2m1, scale e4m3, a block 16 values along the head.
// A code (2 significant bits) times a scale (4) is exact in half precision, whatever both are, so the tensor core gets
// the keys and values that the bits stand for, in f16; the units (powers of two) are factors of the scores and of the
// rows.  Queries: f16 as they are; bf16 ones as f16 relative to the power of two at the row's largest value, which is
// exact down to 2^-14 of it and loses 2^-25 of it at most below that.  Probabilities are rounded to f16, up to
// 2^14 (see kFp4Shift): 2^-11 relative (half a unit of 11 bits) down to 2^-20 of the reference.  Statistics and O are fp32.
//
// The products are transposed, S^T = K Q^T and O^T = V^T P^T: what is wide is the keys and the head, so they take
// the tensor core's 16 rows, and the few query rows its 8 columns.
//
// Tiles: 128 keys, of which every warp takes 32 for itself: it looks up their pages, copies them into a ring of its own
// and works on them, so nothing in the loop waits for another warp.  A lane reads from shared memory just the bytes
// whose values it hands to the tensor core: the order of the values in a contraction is free, so a lane's 4 of every
// 16 are 32 consecutive values of a key, 16 bytes (the queries are laid out to match), and its rows of O^T are 16
// consecutive values.  For V^T two keys' nibbles are brought together in a byte before the conversion, which then
// gives the pair that the tensor core wants.
//
// Bound: HBM (0.56 bytes a value) and, beside it, the conversions: two of every five instructions are e2m1 conversions and
// the products with the scales (ALU 59 %, issue 63 %).  Measured, heads 32/8 of 128, bf16: 64 single tokens ragged to
// 16384 keys (686 MB) 129 us, 5.3 TB/s, 78 % of the measured copy (the bf16 cache of that length is 2.4 GB).  On the way:
// queries on the 16 rows and 64-bit offsets 260, S^T and O^T 144, the warp's maximum only where a lane has outgrown the
// reference 129.  Four CTAs an SM instead of three 133, four stages 131.
// 64 single tokens ragged to 8192 keys, floor and time: heads of 64 25, 50-54 us, of 128 49, 71-75, of 256 102, 128-133.  Other
// heads, and strides that are not whole pieces, go through the loose reads below (8 bytes of codes, scales one by one and
// waited for): 80 35, 134-138, 96 35, 113-117, 112 42, 118-123, 192 74, 243-248.
// Tiles of 32 rows with heads of 128 have 255 registers a thread and spill 280 bytes of stores and 116 of loads, tiles of 16
// rows with heads of 256 (bf16) 8 and 8; the others none.
#pragma once

#include "attention_mma.cuh"

namespace sv {

constexpr int kFp4BN = 128;         // keys of a tile
constexpr int kFp4WarpKeys = 32;    // of which a warp takes this many
// Probabilities are 2^kShift times the weights against the reference, which lie between 0 and 2^kGrow.
constexpr float kFp4Shift = 6.f, kFp4Grow = 8.f;
// Least factor of a row's scores (softmax scale, unit, the queries' power of two): a smaller one, or zero, would make NaN of
// -inf.  The products that it stands before are below 2^36 (256 x 65504 x 2688), so the scores are zero to fp32 either way.
constexpr float kFp4Least = 1e-30f;

template <int DP, int NQ>
struct AttnFp4Geom {
  static constexpr int kRow = DP / 2, kScale = DP / 16;   // bytes of a key's codes and scales
  static constexpr int kCodes = kFp4WarpKeys * kRow, kScales = kFp4WarpKeys * kScale;
  static constexpr int kStage = 2 * (kCodes + kScales);   // one warp's K codes, V codes, K scales, V scales
  static constexpr int kStages = DP == 256 ? 2 : DP == 128 ? 3 : 4;
  static constexpr int kRing = 4 * kStages * kStage, kOut = 4 * 8 * NQ * DP * 4;   // the rows are staged over the ring
  static constexpr int kArea = kRing > kOut ? kRing : kOut;
  static constexpr bool kQSmem = NQ > 2;                  // query fragments of 32 rows have no room in registers
  static constexpr int kSmem = kArea + (kQSmem ? NQ * (DP / 16) * 32 * 8 : 0);
};

// Byte offset of 16-byte piece c of key r in a warp's tile of codes.  The pieces are permuted so that the
// lanes of one read phase fall on distinct banks: K, two keys of four lanes each; V, four keys two apart of two pieces each.
template <int DP>
__device__ __forceinline__ uint32_t fp4_k_piece(int r, int c) {
  return static_cast<uint32_t>(r * (DP / 2) + ((DP == 256 ? c ^ ((r & 1) << 2) : c) << 4));
}
template <int DP>
__device__ __forceinline__ uint32_t fp4_v_piece(int r, int c) {
  constexpr int per = 256 / DP;                      // keys of a 128-byte line
  const int line = r / per, in = r % per * (DP / 32) + c;
  const int x = DP == 64 ? (line & 1) << 1 : DP == 128 ? (line & 3) << 1 : ((r >> 1) & 3) << 1;
  return static_cast<uint32_t>(line * 128 + ((in ^ x) << 4));
}

// Four bytes of two codes each -> four pairs of f16 (low nibble first).
__device__ __forceinline__ void fp4_pairs(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
// Two e4m3 scales -> two f16.
__device__ __forceinline__ uint32_t fp4_scales(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 s;\n\tcvt.u16.u32 s, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, s;\n\t}" : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// For queries of bf16 whose largest magnitude in a row is `top`: the power of two that is taken out (2^k <= top < 2^(k+1)),
// *down its reciprocal.
__device__ __forceinline__ float fp4_query_power(float top, float* down) {
  const int e = max(1, min(static_cast<int>(__float_as_uint(top) >> 23), 253));
  *down = top > 0.f ? __uint_as_float(static_cast<uint32_t>(254 - e) << 23) : 1.f;
  return top > 0.f ? __uint_as_float(static_cast<uint32_t>(e) << 23) : 1.f;
}
template <int N>
__device__ __forceinline__ void cp_async_some(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? N : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(n) : "memory");
}

// 8 x 8 values of 16 bits, transposed across the warp.
__device__ __forceinline__ uint32_t transposed(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}

// NQ: 8-row tiles of queries.
template <bool BF16, int DP, int NQ>
__global__ void __launch_bounds__(kAttnThreads) attn_fp4_kernel(const AttnParams p) {
  using A = AttnType<BF16>;
  using H = AttnType<false>;   // the products are of f16 values
  using Geo = AttnFp4Geom<DP, NQ>;
  constexpr int BM = 8 * NQ, BN = kFp4BN, WK = kFp4WarpKeys, MK = WK / 16, MD = DP / 16, STAGES = Geo::kStages;
  constexpr int WORDS = DP / 32;         // words of 8 codes that a lane reads of a key, of K
  static_assert(MK == 2, "the maximum is written out for 32 keys a warp");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ AttnSchedSmem<kAttnThreads> sched;
  __shared__ float s_ml[4][BM][2];
  __shared__ float s_factor[Geo::kQSmem ? BM : 1];
  float* s_o = reinterpret_cast<float*>(smem);   // [4][BM][DP] after the last key tile
  uint4* s_q = reinterpret_cast<uint4*>(smem + Geo::kArea);   // [DP / 32][NQ][32]: a word's two steps of every lane

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const AttnSplit split = attn_split<BN, true>(p, BM, sched);
  const int cta = blockIdx.x;
  asm volatile("griddepcontrol.launch_dependents;");
  if (cta >= split.n) {
    if (tid == 0) attn_leave_join(p, split, cta, BM, nullptr, false);
    return;
  }
  const long long u_begin = split.begin(cta), u_end = split.begin(cta + 1);
  AttnCursor cur = attn_locate<BN, true>(p, BM, u_begin, sched);
  int k0, k1;
  cur.share(p, u_begin, u_end, &k0, &k1);
  if (k1 <= k0) {   // nothing but an item's overhead
    if (tid == 0) attn_leave_join(p, split, cta, BM, nullptr, false);
    return;
  }
  bool later = false;   // not the CTA's first item
  const uint32_t ring = smem_addr(smem) + warp * STAGES * Geo::kStage;
  const int D = p.c.D, P = p.c.page_size;
  const bool whole = p.s.whole && p.s.alike;   // keys and values in 16-byte pieces, all from one 32-bit offset
  // where this lane reads in a tile: its part of key g and of keys 2 t and 2 t + 1; the other keys follow 8 and 16 keys
  // behind, at the same place of the pieces' permutation
  constexpr int R8 = 8 * Geo::kRow;
  const uint32_t k_at = fp4_k_piece<DP>(g, DP == 64 ? t >> 1 : t) + (DP == 64 ? (t & 1) * 8 : 0);
  const uint32_t k_at1 = DP == 256 ? fp4_k_piece<DP>(g, 4 + t) : 0;
  const uint32_t ks_at = g * Geo::kScale + (DP == 64 ? t : t * 2);
  const int vc = DP == 64 ? g >> 2 : DP == 128 ? g >> 1 : g, vb = DP == 64 ? (g & 3) * 4 : DP == 128 ? (g & 1) * 8 : 0;
  const uint32_t v_at[2] = {fp4_v_piece<DP>(2 * t, vc) + vb, fp4_v_piece<DP>(2 * t + 1, vc) + vb};
  const uint32_t vs_at = 2 * t * Geo::kScale + (DP == 64 ? g >> 1 : DP == 128 ? g : g * 2);

  while (true) {
    const int len = k1 - k0;
    const int rows = cur.req.nq * p.G, r0 = cur.t * BM, r1 = min(rows, r0 + BM);
    int lo, hi;
    attn_keys(p, cur.req, r0, r1, &lo, &hi);
    const int32_t* table = p.c.table + static_cast<long long>(cur.b) * p.c.table_stride;

    auto tile = [&](int j) { return cur.template tile<true>(k0 + j); };   // the CTA's tile number j of the item
    // page of this lane's key of tile j (below 0: nothing to read) and its slot
    auto page_of = [&](int j, int* in) -> int {
      const int key = tile(j) * BN + warp * WK + lane;
      *in = -1;
      if (j >= len || (key < lo && key >= p.sinks) || key >= hi) return -1;   // also what lies before the window
      // key / P: the product with floor(2^32 / P) is the quotient or one less
      int col = static_cast<int>(__umulhi(static_cast<unsigned>(key), p.page_inv));
      *in = key - col * P;
      if (*in >= P) {
        ++col;
        *in -= P;
      }
      return __ldg(table + col);
    };
    // copies of tile j, whose page ids are there
    auto load_tile = [&](int j, uint32_t st, int pg, int in) {
      if (j < len) {
        const bool has = pg >= 0 && pg < p.c.pages && in >= 0;
        if (in >= 0 && !has) atomicOr(p.status, kStatusPageRange);
        const uint32_t dks = st + 2 * Geo::kCodes + lane * Geo::kScale, dvs = dks + Geo::kScales;
        if (whole) {
          const uint32_t at = has ? static_cast<uint32_t>(pg) * static_cast<uint32_t>(p.s.k_page) +
                                        static_cast<uint32_t>(in) * static_cast<uint32_t>(p.s.k_token) +
                                        static_cast<uint32_t>(cur.h) * static_cast<uint32_t>(p.s.k_head)
                                  : 0u;
          const unsigned there = __ballot_sync(0xffffffffu, has);
          constexpr int CH = DP / 32;        // 16-byte pieces of a key
          const int c = lane % CH;
          const uint8_t *kc = p.c.k + c * 16, *vc = p.c.v + c * 16;
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            const int r = i * (32 / CH) + lane / CH;
            const unsigned long long off = static_cast<unsigned long long>(__shfl_sync(0xffffffffu, at, r)) * 8;
            const bool ok = there >> r & 1;
            cp_async16(st + fp4_k_piece<DP>(r, c), kc + off, ok);
            cp_async16(st + Geo::kCodes + fp4_v_piece<DP>(r, c), vc + off, ok);
          }
          cp_async_some<Geo::kScale>(dks, p.s.k + at, has);
          cp_async_some<Geo::kScale>(dvs, p.s.v + at, has);
        } else {                             // heads that are not DP values long, or other strides: 8 bytes, scales one by one
          const long long pl = has ? pg : 0, il = has ? in : 0;
          const uint8_t* k = p.c.k + pl * p.c.k_page + il * p.c.k_token + cur.h * p.c.k_head;
          const uint8_t* v = p.c.v + pl * p.c.v_page + il * p.c.v_token + cur.h * p.c.v_head;
          const uint8_t* ks = p.s.k + pl * p.s.k_page + il * p.s.k_token + cur.h * p.s.k_head;
          const uint8_t* vs = p.s.v + pl * p.s.v_page + il * p.s.v_token + cur.h * p.s.v_head;
          for (int c = 0; c < DP / 16; ++c) {
            const bool ok = has && c * 16 < D;
            cp_async_some<8>(st + fp4_k_piece<DP>(lane, c >> 1) + (c & 1) * 8, ok ? k + c * 8 : k, ok);
            cp_async_some<8>(st + Geo::kCodes + fp4_v_piece<DP>(lane, c >> 1) + (c & 1) * 8, ok ? v + c * 8 : v, ok);
            const uint32_t a = ok ? __ldg(ks + c) : 0u, b = ok ? __ldg(vs + c) : 0u;
            asm volatile("st.shared.u8 [%0], %1;" ::"r"(dks + c), "r"(a) : "memory");
            asm volatile("st.shared.u8 [%0], %1;" ::"r"(dvs + c), "r"(b) : "memory");
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };

    // the first tiles' copies
    int pg_next, in_next;
    {
      int pg[STAGES], in[STAGES];
#pragma unroll
      for (int j = 0; j < STAGES; ++j) pg[j] = page_of(j, &in[j]);
#pragma unroll
      for (int j = 0; j < STAGES - 1; ++j) load_tile(j, ring + j * Geo::kStage, pg[j], in[j]);
      pg_next = pg[STAGES - 1];
      in_next = in[STAGES - 1];
    }

    // query fragments: row g of every 8, step s takes this lane's values 4 s .. 4 s + 3
    uint32_t qf[Geo::kQSmem ? 1 : NQ][DP / 16][2];
    float factor[NQ][2];   // of the scores of rows 2 t and 2 t + 1: softmax scale, the keys' unit, the queries' power of two
    auto fragments = [&](int n, uint32_t (&f)[DP / 16][2]) -> float {
      const int r = r0 + n * 8 + g;
      const uint8_t* q = nullptr;
      if (r < r1) {
        const int tok = attn_token(p, r);
        q = p.q + ((cur.req.q0 + tok) * p.q_token + (cur.h * p.G + r - tok * p.G) * p.q_head) * 2;
      }
      float top = 0.f;
#pragma unroll
      for (int w = 0; w < WORDS; ++w) {
        const int d = DP == 64 ? t * 16 + w * 8 : (w / 4) * 128 + t * 32 + (w % 4) * 8;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (q && d < D) x = __ldg(reinterpret_cast<const uint4*>(q + d * 2));
        f[2 * w][0] = x.x;
        f[2 * w][1] = x.y;
        f[2 * w + 1][0] = x.z;
        f[2 * w + 1][1] = x.w;
        if (BF16) {
          const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(v[e] << 16)), fabsf(__uint_as_float(v[e] & 0xffff0000u))));
        }
      }
      // a negative scale turns the query's sign: the factors are positive
      float mine = fabsf(p.scale_log2);
      if (p.scale_log2 < 0.f) {
#pragma unroll
        for (int s = 0; s < DP / 16; ++s) {
          f[s][0] ^= 0x80008000u;
          f[s][1] ^= 0x80008000u;
        }
      }
      if (BF16) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        float down;
        mine *= fp4_query_power(top, &down);
#pragma unroll
        for (int s = 0; s < DP / 16; ++s)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            f[s][h] = H::pack(__uint_as_float(f[s][h] << 16) * down, __uint_as_float(f[s][h] & 0xffff0000u) * down);
      }
      return fmaxf(mine, kFp4Least);
    };
    if constexpr (Geo::kQSmem) {   // a warp each 8 rows, for all
      static_assert(NQ <= 4, "a warp each");
      if (warp < NQ) {
        const float mine = fragments(warp, qf[0]);
#pragma unroll
        for (int i = 0; i < WORDS; ++i)
          s_q[(i * NQ + warp) * 32 + lane] = make_uint4(qf[0][2 * i][0], qf[0][2 * i][1], qf[0][2 * i + 1][0], qf[0][2 * i + 1][1]);
        if (t == 0) s_factor[warp * 8 + g] = mine;
      }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) factor[n][c] = s_factor[n * 8 + 2 * t + c];
    } else {
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const float mine = fragments(n, qf[n]);
#pragma unroll
        for (int c = 0; c < 2; ++c) factor[n][c] = __shfl_sync(0xffffffffu, mine, (2 * t + c) * 4);
      }
    }
    // key range of this lane's rows
    int row_lo[NQ][2], row_hi[NQ][2], w_lo = 0, w_hi = 0x7fffffff;
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = r0 + n * 8 + 2 * t + c;
        row_lo[n][c] = 0;
        row_hi[n][c] = 0;
        if (r >= r1) continue;
        attn_keys(p, cur.req, r, r + 1, &row_lo[n][c], &row_hi[n][c]);
        w_lo = max(w_lo, row_lo[n][c]);
        w_hi = min(w_hi, row_hi[n][c]);
      }
    // keys inside [w_lo, w_hi) need no mask for any row of the tile (rows that do not exist are not written)
    w_hi = __reduce_min_sync(0xffffffffu, w_hi);
    w_lo = __reduce_max_sync(0xffffffffu, w_lo);

    float o[NQ][MD][4];
    float m[NQ][2], l[NQ][2];   // reference so far, sum of 2^(s - reference + shift)
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
#pragma unroll
      for (int i = 0; i < MD; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[n][i][k] = 0.f;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        m[n][c] = ninf();
        l[n][c] = 0.f;
      }
    }

    uint32_t sk = ring, free = ring + (STAGES - 1) * Geo::kStage;   // the tile to work on, the slot to fill
    for (int j = 0; j < len; ++j) {
      asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
      __syncwarp();
      load_tile(j + STAGES - 1, free, pg_next, in_next);
      pg_next = page_of(j + STAGES, &in_next);

      // S^T = K Q^T: this warp's 32 keys x the rows
      float s[NQ][MK][4];
      uint32_t w[MK][2][WORDS], f[MK][2][DP == 64 ? 1 : WORDS / 2];   // keys g and g + 8 of 16: codes, scales of blocks (twice each)
#pragma unroll
      for (int mk = 0; mk < MK; ++mk) {
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[n][mk][k] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t at = sk + (2 * mk + e) * R8, ks = sk + ks_at + 2 * Geo::kCodes + (2 * mk + e) * 8 * Geo::kScale;
          uint32_t sc;
          if constexpr (DP == 64) {
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[mk][e][0]), "=r"(w[mk][e][1]) : "r"(at + k_at));
            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(sc) : "r"(ks));
            const uint32_t two = fp4_scales(sc);
            f[mk][e][0] = __byte_perm(two, two, 0x1010);
          } else {
#pragma unroll
            for (int h = 0; h < DP / 128; ++h) {
              asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(w[mk][e][4 * h]), "=r"(w[mk][e][4 * h + 1]), "=r"(w[mk][e][4 * h + 2]), "=r"(w[mk][e][4 * h + 3])
                           : "r"(at + (h ? k_at1 : k_at)));
              asm volatile("ld.shared.u16 %0, [%1];" : "=r"(sc) : "r"(ks + h * 8));
              const uint32_t two = fp4_scales(sc);
              f[mk][e][2 * h] = __byte_perm(two, two, 0x1010);
              f[mk][e][2 * h + 1] = __byte_perm(two, two, 0x3232);
            }
          }
        }
      }
      auto add_word = [&](int mk, int i, const uint4 (&q)[NQ]) {
        uint32_t b[2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          fp4_pairs(w[mk][e][i], b[e]);
#pragma unroll
          for (int k = 0; k < 4; ++k) b[e][k] = mul2(b[e][k], f[mk][e][DP == 64 ? 0 : i / 2]);
        }
        const uint32_t a0[4] = {b[0][0], b[1][0], b[0][1], b[1][1]}, a1[4] = {b[0][2], b[1][2], b[0][3], b[1][3]};
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          H::mma(s[n][mk], a0, q[n].x, q[n].y);
          H::mma(s[n][mk], a1, q[n].z, q[n].w);
        }
      };
      if constexpr (Geo::kQSmem) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
          uint4 q[NQ];
#pragma unroll
          for (int n = 0; n < NQ; ++n) q[n] = s_q[(i * NQ + n) * 32 + lane];
#pragma unroll
          for (int mk = 0; mk < MK; ++mk) add_word(mk, i, q);
        }
      } else {
#pragma unroll
        for (int mk = 0; mk < MK; ++mk)
#pragma unroll
          for (int i = 0; i < WORDS; ++i) {
            uint4 q[NQ];
#pragma unroll
            for (int n = 0; n < NQ; ++n) q[n] = make_uint4(qf[n][2 * i][0], qf[n][2 * i][1], qf[n][2 * i + 1][0], qf[n][2 * i + 1][1]);
            add_word(mk, i, q);
          }
      }

      // masks, reference and sum; P^T as the second product's operand
      const int key0 = tile(j) * BN + warp * WK;
      const bool masked = key0 + WK > w_hi || key0 < w_lo;
      if (masked) {
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int mk = 0; mk < MK; ++mk)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = key0 + mk * 16 + (e >> 1) * 8 + g, c = e & 1;
              if (!((key >= row_lo[n][c] || key < p.sinks) && key < row_hi[n][c])) s[n][mk][e] = ninf();
            }
      }
      float mx[NQ][2];   // of this lane's keys: the warp's is wanted only where one of them has outgrown the reference
      bool grow = false;
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          mx[n][c] = fmaxf(fmaxf(s[n][0][c], s[n][0][2 + c]), fmaxf(s[n][1][c], s[n][1][2 + c])) * factor[n][c];
          grow = grow || mx[n][c] - m[n][c] > kFp4Grow;
        }
      if (__any_sync(0xffffffffu, grow)) {   // (the first keys too)
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float top = fmaxf(m[n][c], mx[n][c]);
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            const float f = ex2(m[n][c] - (top == ninf() ? 0.f : top));
            l[n][c] *= f;
            m[n][c] = top;
#pragma unroll
            for (int d = 0; d < MD; ++d) {
              o[n][d][c] *= f;
              o[n][d][2 + c] *= f;
            }
          }
      }
      uint32_t pt[NQ][MK][2];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const float ref[2] = {kFp4Shift - (m[n][0] == ninf() ? 0.f : m[n][0]), kFp4Shift - (m[n][1] == ninf() ? 0.f : m[n][1])};
#pragma unroll
        for (int mk = 0; mk < MK; ++mk)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x = ex2(fmaf(s[n][mk][2 * e], factor[n][0], ref[0])), y = ex2(fmaf(s[n][mk][2 * e + 1], factor[n][1], ref[1]));
            l[n][0] += x;
            l[n][1] += y;
            pt[n][mk][e] = transposed(H::pack(x, y));
          }
      }

      // O^T += V^T P^T
#pragma unroll
      for (int k = 0; k < MK; ++k) {
        constexpr int VW = DP / 64;   // words of 8 codes of a key that are this lane's rows
        uint32_t w[4][VW], f[2][DP == 256 ? 2 : 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t at = sk + v_at[i & 1] + Geo::kCodes + (2 * k + (i >> 1)) * R8;
          if constexpr (DP == 64)
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[i][0]) : "r"(at));
          else if constexpr (DP == 128)
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[i][0]), "=r"(w[i][1]) : "r"(at));
          else
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3])
                         : "r"(at));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {   // scales of the keys 2 t + 8 i and the next one
          const uint32_t at = sk + vs_at + 2 * Geo::kCodes + Geo::kScales + (2 * k + i) * 8 * Geo::kScale;
          uint32_t x, y;
          if constexpr (DP == 256) {
            asm volatile("ld.shared.u16 %0, [%1];" : "=r"(x) : "r"(at));
            asm volatile("ld.shared.u16 %0, [%1];" : "=r"(y) : "r"(at + Geo::kScale));
            f[i][0] = fp4_scales(__byte_perm(x, y, 0x0040));
            f[i][1] = fp4_scales(__byte_perm(x, y, 0x0051));
          } else {
            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(x) : "r"(at));
            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(y) : "r"(at + Geo::kScale));
            f[i][0] = fp4_scales(x | y << 8);
          }
        }
#pragma unroll
        for (int v = 0; v < VW; ++v) {
          const int blk = DP == 256 ? v / 2 : 0;
          uint32_t even[2][4], odd[2][4];   // values 0, 2, 4, 6 and 1, 3, 5, 7 of the word, pairs of keys
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t x = w[2 * i][v], y = w[2 * i + 1][v];
            fp4_pairs((x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u), even[i]);
            fp4_pairs(((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u), odd[i]);
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t a[4] = {mul2(even[0][c], f[0][blk]), mul2(odd[0][c], f[0][blk]), mul2(even[1][c], f[1][blk]),
                                   mul2(odd[1][c], f[1][blk])};
#pragma unroll
            for (int n = 0; n < NQ; ++n) H::mma(o[n][v * 4 + c], a, pt[n][k][0], pt[n][k][1]);
          }
        }
      }
      __syncwarp();   // every lane has read the tile before its slot is filled again
      free = sk;
      sk = sk + Geo::kStage == ring + STAGES * Geo::kStage ? ring : sk + Geo::kStage;
    }

    // join the warps' shares of the keys and write the rows
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float sum = l[n][c];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        const int r = n * 8 + 2 * t + c;
        if (g == 0) {
          s_ml[warp][r][0] = m[n][c] - kFp4Shift;
          s_ml[warp][r][1] = sum;
        }
        // rows g and g + 8 of the product number d are the values 2 d and 2 d + 1 of this lane's
#pragma unroll
        for (int d = 0; d < MD; d += 2)
          *reinterpret_cast<float4*>(s_o + (warp * BM + r) * DP + g * (DP / 8) + 2 * d) =
              make_float4(o[n][d][c], o[n][d][2 + c], o[n][d + 1][c], o[n][d + 1][2 + c]);
      }
    __syncthreads();
    const bool all = len == cur.count;
    const int slot = 2 * cta + (later ? 1 : 0);
    for (int id = tid; id < BM * (DP / 4); id += kAttnThreads) {
      const int r = id / (DP / 4), d = (id % (DP / 4)) * 4;
      if (r0 + r >= r1 || d >= D) continue;
      float mm = ninf();
#pragma unroll
      for (int w = 0; w < 4; ++w) mm = fmaxf(mm, s_ml[w][r][0]);
      const float ref = mm == ninf() ? 0.f : mm;
      float ll = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = ex2(s_ml[w][r][0] - ref);
        ll += f * s_ml[w][r][1];
        const float4 x = *reinterpret_cast<const float4*>(s_o + (w * BM + r) * DP + d);
        acc.x += f * x.x;
        acc.y += f * x.y;
        acc.z += f * x.z;
        acc.w += f * x.w;
      }
      if (all) {
        const float inv = attn_factor(ll, p.v_unit);
        const int tok = attn_token(p, r0 + r);
        const long long row = static_cast<long long>(cur.req.q0 + tok) * p.Hq + cur.h * p.G + (r0 + r - tok * p.G);
        *reinterpret_cast<uint2*>(p.out + (row * D + d) * 2) =
            make_uint2(A::pack(acc.x * inv, acc.y * inv), A::pack(acc.z * inv, acc.w * inv));
        if (d == 0 && p.lse) p.lse[row] = attn_lse(mm, ll);
      } else {
        const long long row = static_cast<long long>(slot) * BM + r;
        *reinterpret_cast<float4*>(p.part_o + row * D + d) = acc;
        if (d == 0) *reinterpret_cast<float2*>(p.part_ml + row * 2) = make_float2(mm, ll);
      }
    }
    AttnCursor next = cur;
    if (!attn_next<BN, true>(p, BM, u_end, &next)) {
      if (tid == 0) attn_leave_join(p, split, cta, BM, &cur, later);
      break;
    }
    cur = next;
    cur.share(p, u_begin, u_end, &k0, &k1);
    later = true;
    __syncthreads();
  }
}

template <bool BF16>
const void* attn_fp4_fn(int dp, int bm);
inline int attn_fp4_smem(int dp, int bm) {
  if (bm == 8) return dp == 64 ? AttnFp4Geom<64, 1>::kSmem : dp == 128 ? AttnFp4Geom<128, 1>::kSmem : AttnFp4Geom<256, 1>::kSmem;
  if (bm == 32) return dp == 64 ? AttnFp4Geom<64, 4>::kSmem : AttnFp4Geom<128, 4>::kSmem;
  return dp == 64 ? AttnFp4Geom<64, 2>::kSmem : dp == 128 ? AttnFp4Geom<128, 2>::kSmem : AttnFp4Geom<256, 2>::kSmem;
}

}  // namespace sv
