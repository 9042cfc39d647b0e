// Rotary positions of new tokens and the write of keys and values into a paged cache held in 4 bits; what such a cache
// stands for.
//
// The rotation is that of the 16-bit caches (rope_append.cu).  A rotated key is rounded to fp32 and to its type (what a
// 16-bit cache would hold) and then, as the values are, held in blocks of 16 along the head:
//   scale = e4m3 nearest to (largest magnitude / (6 unit)), within [2^-9, 448];  code = e2m1 nearest to x / (scale unit),
// ties to the even code.  A block with a NaN gets the scale NaN; what is beyond 6 x 448 units is held as that.
//
// Codes are whole numbers, so they must not hang on a rounding on the way:
// - x has 11 significant bits at most and scale x unit 4, so a quotient is either exactly on a border between two codes
//   or at least 2^-11 of its size away from it (a border has 3 bits).  x times the reciprocal is off by 1.5 x 2^-23 (the
//   reciprocal's 2^-23, the product's rounding), far less than half a unit of half precision (2^-12 at least); rounding that
//   to half precision (11 bits) lands on the border in the first case and off it in the second.
// - largest / (6 unit) in the same way: a tie of e4m3 has 5 bits, 6 times that 7.
// - a rotated key's fp32 error, (|x| + |y|) 2^-21.5 at most, can move its rounding to 16 bits.  Where both ends of that
//   interval do not give the same scale and codes (1 block in some 10^4), the keys in question are rotated in 64 bits.
//
// Bound: HBM (q read and written, k and v read, 4.5 bits a value written, no reuse) and instructions.  Measured, 8192 tokens,
// 32 + 2 x 8 heads of 128, bf16 (177 MB): 46 us, 3.9 TB/s; heads of 80 45 us; rotated parts that are no whole pieces (40 of
// 80) 209 us.  One token: the host's call.
#include <type_traits>

#include "rope_device.cuh"

namespace sv {

namespace {

constexpr int kFp4MaxTokens = 8;   // tokens per CTA: one warp each finds the request and the slot

// A cache's unit and what a largest magnitude is multiplied with.
struct Unit4 {
  float unit, sixth;   // 1 / (6 unit)
};
// The e4m3 scale (as a byte) of a block whose largest magnitude is `top` (NaN: it has one), and 1 / (scale unit).
__device__ __forceinline__ uint32_t block_scale(float top, const Unit4& u, float* inverse) {
  const __half2 want = __floats2half2_rn(fminf(fmaxf(top * u.sixth, 0.001953125f), 448.f), 0.f);
  uint16_t two;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(two) : "r"(*reinterpret_cast<const uint32_t*>(&want)));
  uint32_t half2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(half2) : "h"(two));
  const float scale = __low2float(*reinterpret_cast<const __half2*>(&half2)) * u.unit;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(*inverse) : "f"(scale));
  return top != top ? 0x7fu : two & 0xffu;
}
// The larger; NaN if either is.
__device__ __forceinline__ float larger(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Codes of two values, the first in the low half of the byte.
__device__ __forceinline__ uint32_t two_codes(float x, float y, float inverse) {
  const float2 q = __half22float2(__floats2half2_rn(x * inverse, y * inverse));
  uint32_t r;
  asm("{\n\t.reg .b8 c;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %1, %2;\n\tcvt.u32.u8 %0, c;\n\t}" : "=r"(r) : "f"(q.y), "f"(q.x));
  return r;
}
// Half a block (the other half is the neighbouring lane's, of the same warp): the block's scale, eight codes.
struct Half {
  uint32_t scale, codes;
};
// Called by the whole warp.
__device__ __forceinline__ Half hold(const float (&x)[8], const Unit4& unit) {
  float top = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) top = larger(top, fabsf(x[i]));
  top = larger(top, __shfl_xor_sync(0xffffffffu, top, 1));
  Half b;
  float inverse;
  b.scale = block_scale(top, unit, &inverse);
  b.codes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) b.codes |= two_codes(x[2 * i], x[2 * i + 1], inverse) << (i * 8);
  return b;
}

// Two values rounded to T, and what they are then.
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16*) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half*) {
  const __half2 r = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float2 unpack2(uint32_t x, __nv_bfloat16*) {
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t x, __half*) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }

template <typename T>
__device__ __forceinline__ float rounded(float x) {
  T y;
  from_f(x, &y);
  return to_f(y);
}
// x cos a - y sin a (turn = -1) or x cos a + y sin a (turn = 1) in 64 bits, rounded to fp32.
__device__ __noinline__ float rotated_exactly(float x, float y, float turn, unsigned long long phase, float factor) {
  double s, c;
  sincospi(static_cast<double>(static_cast<long long>(phase)) * 0x1p-63, &s, &c);
  return __double2float_rn((x * c + static_cast<double>(turn) * y * s) * factor);
}

// Byte offsets of a token's slot in the four arrays (-1: not stored), its position, whether a request has it.
struct Slot {
  long long k, v, ks, vs;
  int pos, has;
};
// One warp: the slot of new token n.
__device__ __forceinline__ Slot slot_of(const RopeParams& p, const Fp4Scales& s, int n, int lane) {
  const int b = request_of(p.c.cu_q, p.c.B, n, lane);
  Slot r = {-1, -1, -1, -1, 0, b >= 0 && b < p.c.B};
  if (r.has) {
    r.pos = __ldg(p.c.kv_lens + b) - (__ldg(p.c.cu_q + b + 1) - n);
    if (r.pos >= 0) {
      const int col = r.pos / p.c.page_size, in = r.pos % p.c.page_size;
      const int pg = col < p.c.table_width ? __ldg(p.c.table + b * p.c.table_stride + col) : -1;
      if (pg < 0 || pg >= p.c.pages) {
        if (lane == 0) atomicOr(p.status, kStatusPageRange);
      } else {
        r.k = pg * p.c.k_page + in * p.c.k_token;
        r.v = pg * p.c.v_page + in * p.c.v_token;
        r.ks = pg * s.k_page + in * s.k_token;
        r.vs = pg * s.v_page + in * s.v_token;
      }
    }
  }
  return r;
}

// The form for whole pieces: the rotated part is whole 16-byte pieces (half layout: each half is), rows are 16-byte aligned.
// A CTA takes `per_cta` tokens: a warp each looks up the slot, the CTA computes the angles once for all heads.  Then each
// thread moves 16-byte pieces of 8 values (a piece and its partner where they turn together), the next one's loads
// issued before the current one's work; two lanes hold a block.  (A thread a block reads and writes every second 16 bytes
// at a time: 80 us for 8192 tokens; all three kinds of heads in one loop: 57.)
// SINGLE: where a block has values of both halves (heads of 80), a thread takes one piece and reads its partner beside it, so
// nothing may be rotated in place.
template <int DTYPE, bool INTERLEAVED, bool SINGLE>
__global__ void __launch_bounds__(kRopeThreads)
    rope_fp4_kernel(const RopeParams p, const Fp4Scales s, const Unit4 k_unit, const Unit4 v_unit, int per_cta) {
  using T = typename RopeType<DTYPE>::T;
  constexpr int PP = INTERLEAVED ? 4 : 8;   // pairs of a unit
  extern __shared__ __align__(16) float2 s_cs[];   // [per_cta][rotary / 2]
  __shared__ Slot slots[kFp4MaxTokens];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n0 = blockIdx.x * per_cta, tokens = min(per_cta, p.c.N - n0);
  const int half = p.rotary / 2, D = p.c.D, Hk = p.c.Hkv;
  const int turn = half / PP;                // rotated units per head
  // quotients of small numbers: floor(n ceil(2^32 / d) / 2^32) is exact while n d < 2^32 (the launch sees to it that
  // both are below 2^16)
  auto inverse = [](int d) { return d > 1 ? 0xffffffffu / static_cast<unsigned>(d) + 1u : 0u; };
  auto quotient = [](int n, unsigned inv) { return inv ? static_cast<int>(__umulhi(static_cast<unsigned>(n), inv)) : n; };
  // strides fit 32 bits here: one wide multiplication per address
  auto at2 = [](int i, long long si, int j, long long sj) {
    return static_cast<long long>(i) * static_cast<int>(si) + static_cast<long long>(j) * static_cast<int>(sj);
  };

  auto widen = [](const uint4& raw, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f(reinterpret_cast<const T*>(&raw)[i]);
  };
  auto store = [](T* to, const float (&x)[8]) {
    uint4 raw;
#pragma unroll
    for (int i = 0; i < 8; ++i) from_f(x[i], reinterpret_cast<T*>(&raw) + i);
    *reinterpret_cast<uint4*>(to) = raw;
  };
  for (int t = warp; t < tokens; t += kRopeThreads / 32) {
    const Slot r = slot_of(p, s, n0 + t, lane);
    if (lane == 0) slots[t] = r;
  }
  __syncthreads();
  for (int i = tid; i < tokens * half; i += kRopeThreads) {
    const int t = i / half, j = i - t * half, e = j % PP;
    const float2 c = phase_cs(p.freq[j] * static_cast<unsigned long long>(static_cast<long long>(slots[t].pos)));
    // two pairs' angles together, then the units side by side: the lanes' 16-byte reads fall on distinct banks
    s_cs[t * half + ((e >> 1) * turn + j / PP) * 2 + (e & 1)] = make_float2(c.x * p.factor, c.y * p.factor);
  }
  __syncthreads();

  // the pieces of all queries, of all keys, of all values
  auto pass = [&](auto what) {
    constexpr int KIND = decltype(what)::value;   // 0: queries, 1: keys, 2: values
    constexpr bool PAIR = KIND < 2 && !INTERLEAVED && !SINGLE;
    const int heads = KIND == 0 ? p.Hq : Hk, per_head = KIND == 2 || SINGLE ? D / 8 : turn + (D - p.rotary) / 8;
    const int units = heads * per_head, total = tokens * units;
    const unsigned inv_units = inverse(units), inv_head = inverse(per_head);
    const T* from = reinterpret_cast<const T*>(KIND == 0 ? p.q : KIND == 1 ? p.k : p.v);
    const long long s_token = KIND == 0 ? p.q_token : KIND == 1 ? p.k_token : p.v_token;
    const long long s_head = KIND == 0 ? p.q_head : KIND == 1 ? p.k_head : p.v_head;
    T* to = reinterpret_cast<T*>(KIND == 0 ? p.q_out : KIND == 1 ? p.k_out : nullptr);
    const long long o_token = KIND == 0 ? p.qo_token : p.ko_token, o_head = KIND == 0 ? p.qo_head : p.ko_head;
    struct Unit {
      uint4 a, b;
      int t, h, at;   // token (-1: none), head, first value
      bool rotate;
    };
    auto load = [&](int u, Unit& x) {
      x.t = -1;
      x.h = x.at = 0;
      x.rotate = false;
      x.a = x.b = make_uint4(0, 0, 0, 0);
      if (u >= total) return;
      x.t = quotient(u, inv_units);
      const int r = u - x.t * units;
      x.h = quotient(r, inv_head);
      const int j = r - x.h * per_head;
      x.rotate = KIND < 2 && (SINGLE ? j * 8 < p.rotary : j < turn);
      x.at = KIND == 2 || SINGLE || x.rotate ? j * 8 : p.rotary + (j - turn) * 8;
      const T* src = from + at2(n0 + x.t, s_token, x.h, s_head) + x.at;
      x.a = __ldg(reinterpret_cast<const uint4*>(src));
      if (PAIR && x.rotate) x.b = __ldg(reinterpret_cast<const uint4*>(src + half));
      if (SINGLE && x.rotate) x.b = __ldg(reinterpret_cast<const uint4*>(x.at < half ? src + half : src - half));
    };
    Unit cur;
    load(tid, cur);
    for (int u0 = 0; u0 < total; u0 += kRopeThreads) {   // the same for the whole block: warps work together below
      Unit next;
      load(u0 + kRopeThreads + tid, next);
      const bool mine = cur.t >= 0 && slots[cur.t].has;
      float a[8], b[8];
      widen(cur.a, a);
      if (PAIR || SINGLE) widen(cur.b, b);
      const bool behind = SINGLE && cur.at >= half;   // in the second half
      if (KIND < 2 && mine && cur.rotate) {
        const float4* cs = reinterpret_cast<const float4*>(s_cs + cur.t * half) + (behind ? cur.at - half : cur.at) / 8;
#pragma unroll
        for (int i = 0; i < PP; i += 2) {
          const float4 w = cs[(i >> 1) * turn];   // cos, sin of pairs i and i + 1
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float c = e ? w.z : w.x, sn = e ? w.w : w.y;
            float& x = INTERLEAVED ? a[2 * (i + e)] : a[i + e];
            float& y = INTERLEAVED ? a[2 * (i + e) + 1] : b[i + e];
            const float x1 = behind ? x * c + y * sn : x * c - y * sn, y1 = y * c + x * sn;
            x = x1;
            if (!SINGLE) y = y1;
          }
        }
      }
      const bool pair = PAIR && cur.rotate;
      if (KIND < 2 && mine && to) {
        T* dst = to + at2(n0 + cur.t, o_token, cur.h, o_head) + cur.at;
        store(dst, a);
        if (pair) store(dst + half, b);
      }
      if constexpr (KIND > 0) {
        const bool held = mine && (KIND == 1 ? slots[cur.t].k : slots[cur.t].v) >= 0;
        const Unit4 unit = KIND == 1 ? k_unit : v_unit;
        const float slack = fabsf(p.factor) * 4.76837158203125e-7f;   // 2^-21
        float a0[8], b0[8];   // as they were: for the error, and for the exact rotation
        widen(cur.a, a0);
        widen(cur.b, b0);
#pragma unroll
        for (int which = 0; which < (PAIR ? 2 : 1); ++which) {
          if (which && !__any_sync(0xffffffffu, pair)) break;
          float (&x)[8] = which ? b : a;
          auto partner = [&](int i) { return INTERLEAVED ? a0[i ^ 1] : which ? a0[i] : b0[i]; };
          auto self = [&](int i) { return which ? b0[i] : a0[i]; };
          uint32_t below[4], above[4], apart = 0;   // both ends of each key's error interval, rounded
          if (KIND == 1) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              float e[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) e[k] = cur.rotate ? (fabsf(self(i + k)) + fabsf(partner(i + k))) * slack : 0.f;
              below[i / 2] = pack2(x[i] - e[0], x[i + 1] - e[1], static_cast<T*>(nullptr));
              above[i / 2] = pack2(x[i] + e[0], x[i + 1] + e[1], static_cast<T*>(nullptr));
              apart |= below[i / 2] ^ above[i / 2];
              const float2 r = unpack2(above[i / 2], static_cast<T*>(nullptr));
              x[i] = r.x;
              x[i + 1] = r.y;
            }
          }
          Half y = hold(x, unit);
          if (KIND == 1 && __any_sync(0xffffffffu, held && apart != 0)) {
            // the smaller and the larger of the two in magnitude: scales rise with the largest magnitude and codes with
            // the value, so if these two make equal blocks, no key between the ends makes another one
            float lo[8], hi[8];
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const float2 l = unpack2(below[i / 2], static_cast<T*>(nullptr)), h = unpack2(above[i / 2], static_cast<T*>(nullptr));
              lo[i] = fabsf(h.x) >= fabsf(l.x) ? l.x : h.x;
              hi[i] = fabsf(h.x) >= fabsf(l.x) ? h.x : l.x;
              lo[i + 1] = fabsf(h.y) >= fabsf(l.y) ? l.y : h.y;
              hi[i + 1] = fabsf(h.y) >= fabsf(l.y) ? h.y : l.y;
            }
            const Half z0 = hold(lo, unit), z1 = hold(hi, unit);
            bool differs = z0.scale != z1.scale || z0.codes != z1.codes;
            differs = __shfl_xor_sync(0xffffffffu, differs, 1) || differs;
            if (__any_sync(0xffffffffu, held && differs)) {
              const unsigned long long pos = held ? static_cast<unsigned long long>(static_cast<long long>(slots[cur.t].pos)) : 0ull;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                // what is not rotated is exact (and has no frequency); a NaN of it is equal to nothing
                if (!held || !differs || !cur.rotate || lo[i] == hi[i]) continue;
                const int k = INTERLEAVED ? cur.at / 2 + i / 2 : (behind ? cur.at - half : cur.at) + i;
                const bool second = INTERLEAVED ? i & 1 : which || behind;
                x[i] = rounded<T>(rotated_exactly(self(i), partner(i), second ? 1.f : -1.f, p.freq[k] * pos, p.factor));
              }
              y = hold(x, unit);
            }
          }
          if (held && (!which || pair)) {
            const int i = cur.at + which * half;
            uint8_t* codes = KIND == 1 ? p.c.k + slots[cur.t].k + cur.h * p.c.k_head : p.c.v + slots[cur.t].v + cur.h * p.c.v_head;
            uint8_t* scales = KIND == 1 ? s.k + slots[cur.t].ks + cur.h * s.k_head : s.v + slots[cur.t].vs + cur.h * s.v_head;
            *reinterpret_cast<uint32_t*>(codes + i / 2) = y.codes;
            if (i % 16 == 0) scales[i / 16] = static_cast<uint8_t>(y.scale);
          }
        }
      }
      cur = next;
    }
  };
  pass(std::integral_constant<int, 2>());
  pass(std::integral_constant<int, 1>());
  pass(std::integral_constant<int, 0>());
}

// Any rotated part, alignment and stride of the new tokens: a warp takes a head of a token, a lane every 32nd value, 16 lanes
// a block.  The head is read whole before anything of it is written, so it may be rotated in place.
template <int DTYPE>
__global__ void __launch_bounds__(kRopeThreads)
    rope_fp4_scalar_kernel(const RopeParams p, const Fp4Scales s, const Unit4 k_unit, const Unit4 v_unit) {
  using T = typename RopeType<DTYPE>::T;
  extern __shared__ float2 s_angles[];   // [rotary / 2]
  const int n = blockIdx.x, lane = threadIdx.x & 31;
  const Slot slot = slot_of(p, s, n, lane);
  if (!slot.has) return;   // the same for the whole block
  const int half = p.rotary / 2, D = p.c.D;
  const unsigned long long pos = static_cast<unsigned long long>(static_cast<long long>(slot.pos));
  for (int j = threadIdx.x; j < half; j += kRopeThreads) {
    const float2 w = phase_cs(p.freq[j] * pos);
    s_angles[j] = make_float2(w.x * p.factor, w.y * p.factor);
  }
  __syncthreads();
  for (int h = threadIdx.x / 32; h < p.Hq + 2 * p.c.Hkv; h += kRopeThreads / 32) {
    const int kind = h < p.Hq ? 0 : h < p.Hq + p.c.Hkv ? 1 : 2;   // query, key, value
    const int hk = kind == 0 ? h : kind == 1 ? h - p.Hq : h - p.Hq - p.c.Hkv;
    const T* src = kind == 0   ? reinterpret_cast<const T*>(p.q) + n * p.q_token + hk * p.q_head
                   : kind == 1 ? reinterpret_cast<const T*>(p.k) + n * p.k_token + hk * p.k_head
                               : reinterpret_cast<const T*>(p.v) + n * p.v_token + hk * p.v_head;
    float x[8], self[8], partner[8];   // rotated; as they were
    auto rotated = [&](int c) { return kind < 2 && c < p.rotary; };
    auto pair = [&](int c) { return p.interleaved ? c / 2 : c % half; };
    auto second = [&](int c) { return p.interleaved ? (c & 1) != 0 : c >= half; };
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = i * 32 + lane, with = !rotated(c) ? c : p.interleaved ? c ^ 1 : second(c) ? c - half : c + half;
      self[i] = c < D ? to_f(src[c]) : 0.f;
      partner[i] = c < D ? to_f(src[with]) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = i * 32 + lane;
      x[i] = self[i];
      if (!rotated(c)) continue;
      const float2 w = s_angles[pair(c)];
      x[i] = second(c) ? self[i] * w.x + partner[i] * w.y : self[i] * w.x - partner[i] * w.y;
    }
    __syncwarp();
    T* dst = kind == 0 ? reinterpret_cast<T*>(p.q_out) + n * p.qo_token + hk * p.qo_head
             : kind == 1 && p.k_out ? reinterpret_cast<T*>(p.k_out) + n * p.ko_token + hk * p.ko_head : nullptr;
    const bool held = kind == 1 ? slot.k >= 0 : kind == 2 && slot.v >= 0;
    uint8_t* codes = kind == 1 ? p.c.k + slot.k + hk * p.c.k_head : p.c.v + slot.v + hk * p.c.v_head;
    uint8_t* scales = kind == 1 ? s.k + slot.ks + hk * s.k_head : s.v + slot.vs + hk * s.v_head;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = i * 32 + lane;
      if (dst && c < D) from_f(x[i], dst + c);
      if (!held || i * 32 >= D) continue;     // the same for the whole warp
      const Unit4& unit = kind == 1 ? k_unit : v_unit;
      float inverse;
      auto scale_of = [&](float v) {          // of the 16 lanes' block
        float top = fabsf(v);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) top = larger(top, __shfl_xor_sync(0xffffffffu, top, o));
        return block_scale(top, unit, &inverse);
      };
      float y = rounded<T>(x[i]);
      if (kind == 1) {   // both ends of the error interval, as in the other form
        const float e = rotated(c) ? (fabsf(self[i]) + fabsf(partner[i])) * fabsf(p.factor) * 4.76837158203125e-7f : 0.f;   // 2^-21
        const float below = rounded<T>(x[i] - e), above = rounded<T>(x[i] + e);
        if (__any_sync(0xffffffffu, below != above)) {
          const bool up = fabsf(above) >= fabsf(below);
          const float large = up ? above : below, small = up ? below : above;
          const uint32_t s0 = scale_of(small), c0 = two_codes(small, 0.f, inverse);
          const uint32_t s1 = scale_of(large), c1 = two_codes(large, 0.f, inverse);
          int differs = s0 != s1 || c0 != c1;
#pragma unroll
          for (int o = 1; o < 16; o <<= 1) differs |= __shfl_xor_sync(0xffffffffu, differs, o);
          if (differs && rotated(c) && below != above)   // (a NaN that is not rotated is equal to nothing, and has no frequency)
            y = rounded<T>(rotated_exactly(self[i], partner[i], second(c) ? 1.f : -1.f, p.freq[pair(c)] * pos, p.factor));
        }
      }
      const uint32_t scale = scale_of(y);
      const uint32_t two = two_codes(y, __shfl_down_sync(0xffffffffu, y, 1), inverse);
      if (c < D && lane % 2 == 0) codes[c / 2] = static_cast<uint8_t>(two);
      if (c < D && lane % 16 == 0) scales[c / 16] = static_cast<uint8_t>(scale);
    }
  }
}

// A warp a token, a lane a block: 8 bytes of codes and a scale -> 16 values, two blocks' loads in flight.  Bound: HBM, 0.56
// bytes read and 2 (or 4) written a value.
template <int DTYPE>
__global__ void __launch_bounds__(256) fp4_values_kernel(const Fp4Values p) {
  using T = typename RopeType<DTYPE>::T;
  const int blocks = p.dim / 16, row = p.heads * blocks, lane = threadIdx.x & 31;   // of a head, of a token
  const long long tokens = static_cast<long long>(p.pages) * p.page_size;
  for (long long token = blockIdx.x * 8ll + threadIdx.x / 32; token < tokens; token += gridDim.x * 8ll) {
    const long long page = token / p.page_size;
    const int in = static_cast<int>(token - page * p.page_size);
    const uint8_t* codes_at = p.codes + page * p.page + in * p.token;
    const uint8_t* scales_at = p.scales + page * p.s_page + in * p.s_token;
    T* out_at = static_cast<T*>(p.out) + token * row * 16;
    for (int r0 = lane; r0 < row; r0 += 64) {
      uint2 codes[2];
      uint16_t sc[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int r = r0 + n * 32;
        if (r >= row) continue;
        const int h = r / blocks, j = r - h * blocks;
        codes[n] = __ldg(reinterpret_cast<const uint2*>(codes_at + h * p.head + j * 8));
        sc[n] = __ldg(scales_at + h * p.s_head + j);
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int r = r0 + n * 32;
        if (r >= row) continue;
        uint32_t half2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(half2) : "h"(sc[n]));
        const float scale = __low2float(*reinterpret_cast<const __half2*>(&half2)) * p.unit;
        __align__(16) T out[16];
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          const uint16_t two = static_cast<uint16_t>((b < 4 ? codes[n].x : codes[n].y) >> (8 * (b & 3)) & 0xffu);
          uint32_t v;
          asm("{\n\t.reg .b8 x;\n\tcvt.u8.u16 x, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, x;\n\t}" : "=r"(v) : "h"(two));
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
          from_f(f.x * scale, out + 2 * b);
          from_f(f.y * scale, out + 2 * b + 1);
        }
        uint4* dst = reinterpret_cast<uint4*>(out_at + r * 16);
#pragma unroll
        for (int k = 0; k < static_cast<int>(sizeof(out) / 16); ++k) dst[k] = reinterpret_cast<const uint4*>(out)[k];
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope_fp4(int dtype, const RopeParams& p, const Fp4Scales& s, float k_unit, float v_unit, int sms,
                            cudaStream_t stream) {
  const Unit4 ku = {k_unit, static_cast<float>(1.0 / (6.0 * k_unit))}, vu = {v_unit, static_cast<float>(1.0 / (6.0 * v_unit))};
  const bool q = p.Hq > 0;   // without queries their pointers and strides are anything
  const long long strides[] = {q ? p.q_token : 0, q ? p.q_head : 0, p.k_token, p.k_head, p.v_token, p.v_head,
                               q ? p.qo_token : 0, q ? p.qo_head : 0, p.k_out ? p.ko_token : 0, p.k_out ? p.ko_head : 0};
  bool whole = p.rotary % (p.interleaved ? 8 : 16) == 0;
  const bool single = !p.interleaved && p.rotary % 32 != 0;
  if (single && ((q && p.q_out == p.q) || p.k_out == p.k)) whole = false;
  for (long long st : strides) whole = whole && st % 8 == 0 && st >= 0 && st < (1ll << 31);
  const long long pieces = (p.Hq + 2ll * p.c.Hkv) * (p.c.D / 8);   // of a token; the kernel's quotients hold up to 2^16
  whole = whole && pieces < (1 << 16);
  const void* bases[] = {q ? p.q : nullptr, p.k, p.v, q ? p.q_out : nullptr, p.k_out};
  for (const void* b : bases) whole = whole && (reinterpret_cast<uintptr_t>(b) & 15) == 0;
  if (!whole) {
    const dim3 grid(p.c.N), block(kRopeThreads);
    const size_t smem = sizeof(float2) * (p.rotary / 2);
    if (dtype == 1) rope_fp4_scalar_kernel<1><<<grid, block, smem, stream>>>(p, s, ku, vu);
    if (dtype == 2) rope_fp4_scalar_kernel<2><<<grid, block, smem, stream>>>(p, s, ku, vu);
    return cudaGetLastError();
  }
  // few tokens: a CTA each; many: as many tokens a CTA as make about 4096 pieces.  8192 tokens of 768 pieces: 1024 pieces
  // 64 us, 2048 48, 4096 46, 6144 53 (too few CTAs for the last wave).
  int per = p.c.N <= 4 * sms ? 1 : static_cast<int>(4096 / pieces);
  per = per < 1 ? 1 : per > kFp4MaxTokens ? kFp4MaxTokens : per;
  const dim3 grid((p.c.N + per - 1) / per), block(kRopeThreads);
  const size_t smem = sizeof(float2) * (p.rotary / 2) * per;
  const int kind = dtype * 4 + (p.interleaved ? 1 : single ? 2 : 0);
  if (kind == 4) rope_fp4_kernel<1, false, false><<<grid, block, smem, stream>>>(p, s, ku, vu, per);
  if (kind == 5) rope_fp4_kernel<1, true, false><<<grid, block, smem, stream>>>(p, s, ku, vu, per);
  if (kind == 6) rope_fp4_kernel<1, false, true><<<grid, block, smem, stream>>>(p, s, ku, vu, per);
  if (kind == 8) rope_fp4_kernel<2, false, false><<<grid, block, smem, stream>>>(p, s, ku, vu, per);
  if (kind == 9) rope_fp4_kernel<2, true, false><<<grid, block, smem, stream>>>(p, s, ku, vu, per);
  if (kind == 10) rope_fp4_kernel<2, false, true><<<grid, block, smem, stream>>>(p, s, ku, vu, per);
  return cudaGetLastError();
}

cudaError_t launch_fp4_values(int dtype, const Fp4Values& p, int sms, cudaStream_t stream) {
  const long long tokens = static_cast<long long>(p.pages) * p.page_size;
  if (tokens == 0) return cudaSuccess;
  const long long want = (tokens + 7) / 8;
  const dim3 grid(static_cast<unsigned>(want < 16ll * sms ? want : 16ll * sms)), block(256);
  if (dtype == 0) fp4_values_kernel<0><<<grid, block, 0, stream>>>(p);
  if (dtype == 1) fp4_values_kernel<1><<<grid, block, 0, stream>>>(p);
  if (dtype == 2) fp4_values_kernel<2><<<grid, block, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace sv
