// Fixed-point softmax weights of the sampling kernel.
//
// A token's weight is 2^((z - max) c), c = log2(e) / T, as an integer in units of 2^-44.  Integer
// sums do not depend on their order, so the cut of top-p and the drawn token are the same whatever
// the split of the work; a row's total stays below 2^62 (V <= 2^18).  The weight's relative error is
// below 2^-36: the draw compares sums with u x total, and an error of fp32's size (2^-23, over 10^5
// boundaries) would move a drawn token in one row of a few hundred.
#pragma once

#include "spec_device.cuh"

namespace sv {

constexpr int kWeightBits = 44;
constexpr unsigned long long kWeightOne = 1ull << kWeightBits;

// 2^(i / 64) x 2^62, rounded.
static __device__ __constant__ unsigned long long kExp2Table[64] = {
    0x4000000000000000ull, 0x40b268f9de0183baull, 0x4166c34c5615d0ecull, 0x421d1461d66f2023ull,
    0x42d561b3e6243d8aull, 0x438fb0cb4f468808ull, 0x444c0740496d4294ull, 0x450a6abaa4b77ecdull,
    0x45cae0f1f545eb73ull, 0x468d6fadbf2dd4f3ull, 0x47521cc5a2e6a9e0ull, 0x4818ee218a3358eeull,
    0x48e1e9b9d588e19bull, 0x49ad159789f37496ull, 0x4a7a77d47f7b84b1ull, 0x4b4a169b900c2d00ull,
    0x4c1bf828c6dc54b8ull, 0x4cf022c9905bfd32ull, 0x4dc69cdceaa72a9cull, 0x4e9f6cd3967fdba8ull,
    0x4f7a993048d088d7ull, 0x50582887dcb8a7e1ull, 0x513821818624b40cull, 0x521a8ad704f3404full,
    0x52ff6b54d8a89c75ull, 0x53e6c9da74b29ab5ull, 0x54d0ad5a753e077cull, 0x55bd1cdad49f699cull,
    0x56ac1f752150a563ull, 0x579dbc56b48521baull, 0x5891fac0e95612c8ull, 0x5988e20954889245ull,
    0x5a827999fcef3242ull, 0x5b7ec8f19468bbc9ull, 0x5c7dd7a3b17dcf75ull, 0x5d7fad59099f22feull,
    0x5e8451cfac061b5full, 0x5f8bccdb3d398841ull, 0x6096266533384a2bull, 0x61a3666d124bb204ull,
    0x62b39508aa836d6full, 0x63c6ba6455dcd8aeull, 0x64dcdec3371793d1ull, 0x65f60a7f79393e2eull,
    0x6712460a8fc24072ull, 0x683199ed779592caull, 0x69540ec8f895722dull, 0x6a79ad55e7f6fd10ull,
    0x6ba27e656b4eb57aull, 0x6cce8ae13c57ebdbull, 0x6dfddbcbed791babull, 0x6f307a412f074892ull,
    0x70666f76154a7089ull, 0x719fc4b95f452d29ull, 0x72dc8373be41a454ull, 0x741cb5281e25ee34ull,
    0x75606373ee921c97ull, 0x76a7980f6cca15c2ull, 0x77f25ccdee6d7ae6ull, 0x7940bb9e2cffd89dull,
    0x7a92be8a92436616ull, 0x7be86fb985689ddcull, 0x7d41d96db915019dull, 0x7e9f06067a4360baull,
};

// One row's scale: c = c_hi + c_lo.
struct WeightScale {
  float zmax, c_hi, c_lo;
};
__device__ __forceinline__ WeightScale weight_scale(float zmax, float T) {
  const double c = 1.4426950408889634 / static_cast<double>(T);
  WeightScale s;
  s.zmax = zmax;
  s.c_hi = static_cast<float>(c);
  s.c_lo = static_cast<float>(c - static_cast<double>(s.c_hi));
  return s;
}

// (z - max) c as a sum of two floats, then as a fixed-point number with 38 fraction bits: n whole
// binary places, 6 bits for the table, 32 bits r for 2^r = 1 + y + y^2/2 + y^3/6 + y^4/24, y = r ln 2 < 0.011.
// `tab`: the table, in shared memory (lanes read different entries).
__device__ __forceinline__ unsigned long long weight_of(float z, const WeightScale& s, const unsigned long long* tab) {
  if (z == s.zmax) return kWeightOne;
  const float dh = z - s.zmax, bb = dh - z;
  const float p = dh * s.c_hi;
  if (!(p >= -48.f)) return 0ull;   // below half a unit (or -inf)
  const float dl = (z - (dh - bb)) + (-s.zmax - bb);
  const float pe = fmaf(dh, s.c_hi, -p) + fmaf(dh, s.c_lo, dl * s.c_hi);
  const long long x = __float2ll_rn(p * 274877906944.f) + __float2int_rn(pe * 274877906944.f);
  const int n = static_cast<int>(x >> 38);
  const unsigned f = static_cast<unsigned>(x >> 32) & 63u, r = static_cast<unsigned>(x);
  const unsigned y38 = __umulhi(r, 0xb17217f8u);                       // y x 2^38; ln 2 x 2^32, rounded
  const float yf = static_cast<float>(y38), y = yf * 3.637978807091713e-12f;
  const float g = y * 0.5f * fmaf(y * 0.3333333433f, fmaf(y, 0.25f, 1.f), 1.f);
  const unsigned s38 = y38 + __float2uint_rn(yf * g);
  const unsigned long long e = tab[f];
  const unsigned long long w =
      e + ((static_cast<unsigned long long>(static_cast<unsigned>(e >> 31)) * s38) >> 7);
  const int sh = 61 - kWeightBits - n;                                  // one bit left for rounding
  return sh >= 63 ? 0ull : ((w >> sh) + 1) >> 1;
}

}  // namespace sv
