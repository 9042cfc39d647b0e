// Attention of new tokens over a paged cache, mma.sync kernel: any page size, head sizes up to 256.
//
//   O = softmax(scale Q K^T + mask) V,  lse = ln sum exp(scale q k)   for every new token and query head
//
// with one pass over the keys: per row the running maximum m and sum l of 2^(s - m) (s in units of
// log 2), O rescaled by 2^(m_old - m) when the maximum grows.  Statistics and O are fp32; the
// probabilities are rounded to the operands' type for the second product, because the tensor core takes no
// wider operand beside values of that type: half a unit of the type in each, the size of the output's own
// rounding.  Relative error against 64 bits, bf16: 0.0019 (one token) to 0.0023 (17 tokens), of which the
// output's rounding alone makes 0.0017.
//
// Tiles: the rows of an item are (token, query head of the key head) pairs, so keys and values are
// read once for all the heads that share them.  16-row tiles (few rows: single tokens) give every
// warp all rows and a quarter of the 64 keys, and join the warps at the end; 64-row tiles give every
// warp 16 rows.  Keys and values come by 16-byte asynchronous copies, row addresses a key tile ahead
// from the page table, in a ring of STAGES tiles; 16-byte pieces are permuted by the row's low bits,
// which makes the matrix loads free of bank conflicts.
//
// Bound: HBM (a key and value byte meets 4 rows x 4 flop at most in its main use).  Measured, heads 32/8 of
// 128, bf16: 64 single tokens over caches ragged to 8192 keys (1.14 GB) 192-195 us, 5.9 TB/s, 86 % of the
// measured copy; 64 x 4 tokens to 4096 keys (634 MB) 111-113 us, 83 %.  What is left is the start, the tail
// and the ring filled anew for every item.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attention_sched.cuh"

namespace sv {

constexpr int kAttnThreads = 128;
constexpr int kAttnBN = 64;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

template <bool BF16>
struct AttnType;
template <>
struct AttnType<true> {
  using T = __nv_bfloat16;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
template <>
struct AttnType<false> {
  using T = __half;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

// Byte offset of 16-byte piece c of row r in a tile of DP-element rows.
template <int DP>
__device__ __forceinline__ uint32_t attn_piece(int r, int c) {
  return static_cast<uint32_t>(r * (DP * 2) + ((c ^ (r & 7)) << 4));
}

template <int DP, int WM>
struct AttnMmaGeom {
  static constexpr bool kQReg = DP <= 128;   // query fragments fit the registers beside O
  static constexpr int kTile = kAttnBN * DP * 2;
  static constexpr int kStages = DP >= 256 ? (WM == 1 ? 3 : 2) : (DP >= 128 ? 3 : 4);
  static constexpr int kRing = kStages + 2;
  static constexpr int kQBytes = kQReg ? 0 : 16 * WM * DP * 2;
  static constexpr int kSmem = kStages * 2 * kTile + kQBytes + kRing * kAttnBN * 16;
};

template <bool BF16, int DP, int WM>
__global__ void __launch_bounds__(kAttnThreads) attn_mma_kernel(const AttnParams p) {
  using A = AttnType<BF16>;
  using Geo = AttnMmaGeom<DP, WM>;
  constexpr int WN = 4 / WM, BM = 16 * WM, BN = kAttnBN, KPW = BN / WN, NT = KPW / 8, DT = DP / 8, KS = DP / 16;
  constexpr int STAGES = Geo::kStages, RING = Geo::kRing;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ AttnSchedSmem<kAttnThreads> sched;
  __shared__ float s_ml[WN][BM][2];
  uint8_t* s_q = smem + STAGES * 2 * Geo::kTile;
  longlong2* s_off = reinterpret_cast<longlong2*>(s_q + Geo::kQBytes);   // [RING][BN] byte offsets of key and value rows
  float* s_o = reinterpret_cast<float*>(smem);                           // [WN][BM][DP] after the last key tile
  static_assert(WN * BM * DP * 4 <= STAGES * 2 * Geo::kTile, "the output staging fits the ring");

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wm = warp / WN, wn = warp % WN;
  const AttnSplit split = attn_split<BN>(p, BM, sched);
  const int cta = blockIdx.x;
  asm volatile("griddepcontrol.launch_dependents;");
  if (cta >= split.n) {
    if (tid == 0) attn_leave_join(p, split, cta, BM, nullptr, false);
    return;
  }
  const long long u_begin = split.begin(cta), u_end = split.begin(cta + 1);
  AttnCursor cur = attn_locate<BN>(p, BM, u_begin, sched);
  int k0, k1;
  cur.share(p, u_begin, u_end, &k0, &k1);
  if (k1 <= k0) {   // nothing but an item's overhead
    if (tid == 0) attn_leave_join(p, split, cta, BM, nullptr, false);
    return;
  }
  bool later = false;   // not the CTA's first item
  const uint32_t smem_base = smem_addr(smem);
  const int D = p.c.D, P = p.c.page_size;

  while (true) {
    const int kt0 = cur.first + k0, len = k1 - k0;
    const int rows = cur.req.nq * p.G, r0 = cur.t * BM, r1 = min(rows, r0 + BM);
    int lo, hi;
    attn_keys(p, cur.req, r0, r1, &lo, &hi);
    const int32_t* table = p.c.table + static_cast<long long>(cur.b) * p.c.table_stride;
    const uint8_t* kbase = p.c.k + static_cast<long long>(cur.h) * p.c.k_head * 2;
    const uint8_t* vbase = p.c.v + static_cast<long long>(cur.h) * p.c.v_head * 2;

    // page id of this thread's key of tile j (-1: nothing to read)
    auto page_of = [&](int j) -> int {
      const int key = (kt0 + j) * BN + (tid & (BN - 1));
      if (j >= len || key < lo || key >= hi) return -1;   // also of the first tile what lies before the window
      const int pg = __ldg(table + key / P);
      if (pg < 0 || pg >= p.c.pages) {
        atomicOr(p.status, kStatusPageRange);
        return -1;
      }
      return pg;
    };
    auto put_offset = [&](int j, int pg) {
      const int key = (kt0 + j) * BN + (tid & (BN - 1));
      const int in = key % P;
      longlong2 o = make_longlong2(-1, -1);
      if (pg >= 0)
        o = make_longlong2((pg * p.c.k_page + in * p.c.k_token) * 2, (pg * p.c.v_page + in * p.c.v_token) * 2);
      s_off[(j % RING) * BN + (tid & (BN - 1))] = o;
    };
    auto load_tile = [&](int j) {
      if (j < len) {
        const uint32_t st = smem_base + (j % STAGES) * 2 * Geo::kTile;
        constexpr int CH = DP / 8;   // pieces per row
#pragma unroll
        for (int i = 0; i < BN * CH / kAttnThreads; ++i) {
          const int id = i * kAttnThreads + tid, r = id / CH, c = id % CH;
          const longlong2 o = s_off[(j % RING) * BN + r];
          const bool ok = o.x >= 0 && c * 8 < D;
          const uint32_t at = st + attn_piece<DP>(r, c);
          cp_async16(at, ok ? kbase + o.x + c * 16 : kbase, ok);
          cp_async16(at + Geo::kTile, ok ? vbase + o.y + c * 16 : vbase, ok);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };

    // row addresses of the first tiles (two tiles at a time: 128 threads, 64 keys), the next ones in registers
#pragma unroll
    for (int j = 0; j < STAGES; j += 2) {
      const int jj = j + tid / BN;
      if (jj < STAGES) put_offset(jj, page_of(jj));
    }
    int pg_next = tid < BN ? page_of(STAGES) : -1;

    // query fragments: rows lane/4 and lane/4 + 8 of the warp's 16
    uint32_t qf[Geo::kQReg ? KS : 1][4];
    auto q_ptr = [&](int r) {
      const int tok = cur.req.q0 + attn_token(p, r), head = cur.h * p.G + r - (attn_token(p, r)) * p.G;
      return p.q + (tok * p.q_token + head * p.q_head) * 2;
    };
    if constexpr (Geo::kQReg) {
      const int ra = r0 + wm * 16 + lane / 4, rb = ra + 8;
      const uint8_t* qa = ra < r1 ? q_ptr(ra) : nullptr;
      const uint8_t* qb = rb < r1 ? q_ptr(rb) : nullptr;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int d = k * 16 + (lane & 3) * 2;
        qf[k][0] = qa && d < D ? __ldg(reinterpret_cast<const uint32_t*>(qa + d * 2)) : 0u;
        qf[k][1] = qb && d < D ? __ldg(reinterpret_cast<const uint32_t*>(qb + d * 2)) : 0u;
        qf[k][2] = qa && d + 8 < D ? __ldg(reinterpret_cast<const uint32_t*>(qa + d * 2 + 16)) : 0u;
        qf[k][3] = qb && d + 8 < D ? __ldg(reinterpret_cast<const uint32_t*>(qb + d * 2 + 16)) : 0u;
      }
    } else {
      for (int id = tid; id < BM * (DP / 8); id += kAttnThreads) {
        const int r = id / (DP / 8), c = id % (DP / 8);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r0 + r < r1 && c * 8 < D) v = __ldg(reinterpret_cast<const uint4*>(q_ptr(r0 + r) + c * 16));
        *reinterpret_cast<uint4*>(s_q + attn_piece<DP>(r, c)) = v;
      }
    }
    // key range of this lane's two rows
    int row_lo[2], row_hi[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + wm * 16 + lane / 4 + i * 8;
      row_lo[i] = 0;
      row_hi[i] = 0;
      if (r < r1) attn_keys(p, cur.req, r, r + 1, &row_lo[i], &row_hi[i]);
    }

    float o[DT][4];
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
    float m[2] = {ninf(), ninf()}, l[2] = {0.f, 0.f};

    __syncthreads();
#pragma unroll
    for (int j = 0; j < STAGES - 1; ++j) load_tile(j);

    for (int j = 0; j < len; ++j) {
      asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
      __syncthreads();
      load_tile(j + STAGES - 1);
      if (tid < BN) {
        put_offset(j + STAGES, pg_next);
        pg_next = page_of(j + STAGES + 1);
      }
      const uint32_t sk = smem_base + (j % STAGES) * 2 * Geo::kTile, sv_ = sk + Geo::kTile;

      // S = Q K^T: this warp's rows x its KPW keys
      float s[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[i][k] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t a[4];
        if constexpr (Geo::kQReg) {
#pragma unroll
          for (int e = 0; e < 4; ++e) a[e] = qf[k][e];
        } else {
          ldsm4(smem_addr(s_q) + attn_piece<DP>(wm * 16 + (lane & 15), k * 2 + (lane >> 4)), a);
        }
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
          uint32_t b[4];
          const int r = wn * KPW + n * 8 + (lane & 7) + ((lane >> 4) << 3);
          ldsm4(sk + attn_piece<DP>(r, k * 2 + ((lane >> 3) & 1)), b);
          A::mma(s[n], a, b[0], b[1]);
          A::mma(s[n + 1], a, b[2], b[3]);
        }
      }

      // masks, running maximum and sum
      const int kb = (kt0 + j) * BN + wn * KPW + (lane & 3) * 2;
      float mx[2] = {m[0], m[1]};
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = kb + n * 8 + (e & 1), i = e >> 1;
          const float x = key >= row_lo[i] && key < row_hi[i] ? s[n][e] * p.scale_log2 : ninf();
          s[n][e] = x;
          mx[i] = fmaxf(mx[i], x);
        }
      float ref[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
        ref[i] = mx[i] == ninf() ? 0.f : mx[i];
        const float f = ex2(m[i] - ref[i]);
        l[i] *= f;
        m[i] = mx[i];
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          o[d][2 * i] *= f;
          o[d][2 * i + 1] *= f;
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[n][e] = ex2(s[n][e] - ref[e >> 1]);
          l[e >> 1] += s[n][e];
        }

      // O += P V
#pragma unroll
      for (int k = 0; k < KPW / 16; ++k) {
        uint32_t a[4] = {A::pack(s[2 * k][0], s[2 * k][1]), A::pack(s[2 * k][2], s[2 * k][3]),
                         A::pack(s[2 * k + 1][0], s[2 * k + 1][1]), A::pack(s[2 * k + 1][2], s[2 * k + 1][3])};
#pragma unroll
        for (int d = 0; d < DT; d += 2) {
          uint32_t b[4];
          const int r = wn * KPW + k * 16 + (lane & 15);
          ldsm4t(sv_ + attn_piece<DP>(r, d + (lane >> 4)), b);
          A::mma(o[d], a, b[0], b[1]);
          A::mma(o[d + 1], a, b[2], b[3]);
        }
      }
    }

    // join the warps' shares of the keys and write the rows
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      const int r = wm * 16 + lane / 4 + i * 8;
      if ((lane & 3) == 0) {
        s_ml[wn][r][0] = m[i];
        s_ml[wn][r][1] = l[i];
      }
#pragma unroll
      for (int d = 0; d < DT; ++d)
        *reinterpret_cast<float2*>(s_o + (wn * BM + r) * DP + d * 8 + (lane & 3) * 2) =
            make_float2(o[d][2 * i], o[d][2 * i + 1]);
    }
    __syncthreads();
    const bool whole = len == cur.count;
    const int slot = 2 * cta + (later ? 1 : 0);
    for (int id = tid; id < BM * (DP / 4); id += kAttnThreads) {
      const int r = id / (DP / 4), d = (id % (DP / 4)) * 4;
      if (r0 + r >= r1 || d >= D) continue;
      float mm = ninf();
#pragma unroll
      for (int w = 0; w < WN; ++w) mm = fmaxf(mm, s_ml[w][r][0]);
      const float ref = mm == ninf() ? 0.f : mm;
      float ll = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WN; ++w) {
        const float f = ex2(s_ml[w][r][0] - ref);
        ll += f * s_ml[w][r][1];
        const float4 x = *reinterpret_cast<const float4*>(s_o + (w * BM + r) * DP + d);
        acc.x += f * x.x;
        acc.y += f * x.y;
        acc.z += f * x.z;
        acc.w += f * x.w;
      }
      if (whole) {
        const float inv = ll > 0.f ? 1.f / ll : 0.f;
        const int tok = attn_token(p, r0 + r);
        const long long row = static_cast<long long>(cur.req.q0 + tok) * p.Hq + cur.h * p.G + (r0 + r - tok * p.G);
        uint2 w = make_uint2(A::pack(acc.x * inv, acc.y * inv), A::pack(acc.z * inv, acc.w * inv));
        *reinterpret_cast<uint2*>(p.out + (row * D + d) * 2) = w;
        if (d == 0 && p.lse) p.lse[row] = ll > 0.f ? (mm + log2f(ll)) * 0.69314718055994531f : ninf();
      } else {
        const long long row = static_cast<long long>(slot) * BM + r;
        *reinterpret_cast<float4*>(p.part_o + row * D + d) = acc;
        if (d == 0) *reinterpret_cast<float2*>(p.part_ml + row * 2) = make_float2(mm, ll);
      }
    }
    AttnCursor next = cur;
    if (!attn_next<BN>(p, BM, u_end, &next)) {
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
const void* attn_mma_fn(int dp, int bm);
template <bool BF16>
int attn_mma_smem(int dp, int bm) {
  if (bm == 16) return dp == 64 ? AttnMmaGeom<64, 1>::kSmem : dp == 128 ? AttnMmaGeom<128, 1>::kSmem : AttnMmaGeom<256, 1>::kSmem;
  return dp == 64 ? AttnMmaGeom<64, 4>::kSmem : dp == 128 ? AttnMmaGeom<128, 4>::kSmem : AttnMmaGeom<256, 4>::kSmem;
}

}  // namespace sv
