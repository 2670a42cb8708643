// hw_rope_exact.cuh - cos and sin of a RoPE angle to within 2^-36, rounded
// to fp32.  Keys that are stored in 4 bits come out the same however they are
// computed only if the rotation before the rounding to codes is: a code step is a
// large part of a value, and one unit in the last place of a cosine moves about one
// key element in 10^7 across a border between codes.
//
// The angle is p * phase mod 2^64 in units of 2^-64 turns, exact.  Its nearest 256th of a
// turn is looked up as two fp32 parts, the rest (at most pi/256) goes through the
// first terms of the Taylor series, in two parts as well, and the two are joined by the
// addition theorem.  About 45 fp32 instructions; fp64 would take as many at 1/64 of
// the rate.
#pragma once

#include <stdint.h>

namespace hw {

// sin(2 pi k / 256) for k = 0 .. 64, as the nearest fp32 and that of the rest.
__device__ const float2 kSin256[65] = {
    {0x0.0p+0f, 0x0.0p+0f}, {0x1.9215600000000p-6f, -0x1.0b93300000000p-31f},
    {0x1.91f6600000000p-5f, -0x1.de44fe0000000p-30f}, {0x1.2d520a0000000p-4f, -0x1.a63cc20000000p-29f},
    {0x1.917a6c0000000p-4f, -0x1.eb25ea0000000p-31f}, {0x1.f564e60000000p-4f, -0x1.2ad19e0000000p-29f},
    {0x1.2c81060000000p-3f, 0x1.d1cc280000000p-28f}, {0x1.5e21440000000p-3f, 0x1.22cff20000000p-29f},
    {0x1.8f8b840000000p-3f, -0x1.cb2cfa0000000p-30f}, {0x1.c0b8260000000p-3f, 0x1.4fc9ec0000000p-28f},
    {0x1.f19f980000000p-3f, -0x1.37a83a0000000p-29f}, {0x1.111d260000000p-2f, 0x1.58fb3c0000000p-29f},
    {0x1.2940620000000p-2f, 0x1.dab3e00000000p-27f}, {0x1.4135ca0000000p-2f, -0x1.7d13400000000p-27f},
    {0x1.58f9a80000000p-2f, -0x1.4a9c040000000p-27f}, {0x1.7088540000000p-2f, -0x1.e0b74c0000000p-27f},
    {0x1.87de2a0000000p-2f, 0x1.abaa580000000p-28f}, {0x1.9ef7940000000p-2f, 0x1.d476c60000000p-29f},
    {0x1.b5d1000000000p-2f, 0x1.3c2b980000000p-27f}, {0x1.cc66ea0000000p-2f, -0x1.b38ee80000000p-28f},
    {0x1.e2b5d40000000p-2f, -0x1.fe42720000000p-28f}, {0x1.f8ba4e0000000p-2f, -0x1.01d9520000000p-28f},
    {0x1.07387a0000000p-1f, -0x1.b740040000000p-27f}, {0x1.11eb360000000p-1f, -0x1.7c969c0000000p-26f},
    {0x1.1c73b40000000p-1f, -0x1.9465ce0000000p-27f}, {0x1.26d0540000000p-1f, 0x1.9ba25c0000000p-26f},
    {0x1.30ff800000000p-1f, -0x1.8f47e60000000p-28f}, {0x1.3affa20000000p-1f, 0x1.240a180000000p-26f},
    {0x1.44cf320000000p-1f, 0x1.4247760000000p-27f}, {0x1.4e6cac0000000p-1f, -0x1.0706860000000p-27f},
    {0x1.57d6940000000p-1f, -0x1.6e626c0000000p-26f}, {0x1.610b760000000p-1f, -0x1.5c5a640000000p-26f},
    {0x1.6a09e60000000p-1f, 0x1.9fcef40000000p-27f}, {0x1.72d0840000000p-1f, -0x1.02000e0000000p-26f},
    {0x1.7b5df20000000p-1f, 0x1.3557d80000000p-28f}, {0x1.83b0e00000000p-1f, 0x1.7ff2ee0000000p-26f},
    {0x1.8bc8060000000p-1f, 0x1.62a2e80000000p-26f}, {0x1.93a2240000000p-1f, 0x1.324c800000000p-26f},
    {0x1.9b3e040000000p-1f, 0x1.fce1d00000000p-27f}, {0x1.a29a7a0000000p-1f, 0x1.189e080000000p-31f},
    {0x1.a9b6620000000p-1f, 0x1.21d4340000000p-26f}, {0x1.b090a60000000p-1f, -0x1.fabf800000000p-27f},
    {0x1.b728340000000p-1f, 0x1.465b900000000p-27f}, {0x1.bd7c0a0000000p-1f, 0x1.8df2a60000000p-26f},
    {0x1.c38b300000000p-1f, -0x1.cfe84a0000000p-26f}, {0x1.c954b20000000p-1f, 0x1.3411f40000000p-29f},
    {0x1.ced7b00000000p-1f, -0x1.7867120000000p-26f}, {0x1.d4134e0000000p-1f, -0x1.d646d80000000p-26f},
    {0x1.d906bc0000000p-1f, 0x1.e651a80000000p-26f}, {0x1.ddb13c0000000p-1f, -0x1.2667b80000000p-26f},
    {0x1.e212100000000p-1f, 0x1.3da1ba0000000p-27f}, {0x1.e6288e0000000p-1f, 0x1.891c220000000p-26f},
    {0x1.e9f4160000000p-1f, -0x1.273a440000000p-26f}, {0x1.ed740e0000000p-1f, 0x1.da12580000000p-27f},
    {0x1.f0a7f00000000p-1f, -0x1.1b73ca0000000p-27f}, {0x1.f38f3a0000000p-1f, 0x1.8c9cb20000000p-26f},
    {0x1.f6297c0000000p-1f, 0x1.feeb960000000p-26f}, {0x1.f876500000000p-1f, -0x1.63ad160000000p-27f},
    {0x1.fa75580000000p-1f, -0x1.eeb5d20000000p-30f}, {0x1.fc26480000000p-1f, -0x1.e3cc060000000p-26f},
    {0x1.fd88da0000000p-1f, 0x1.e892920000000p-28f}, {0x1.fe9cda0000000p-1f, 0x1.a031080000000p-26f},
    {0x1.ff621e0000000p-1f, 0x1.bcb6be0000000p-28f}, {0x1.ffd8860000000p-1f, 0x1.099a1a0000000p-30f},
    {0x1.0000000000000p+0f, 0x0.0p+0f},
};
// 2 pi / 2^64, likewise.
constexpr float kTurnHi = 0x1.921fb60000000p-62f, kTurnLo = -0x1.777a5c0000000p-87f;

// a + b as hi + lo, exactly.
__device__ __forceinline__ float two_sum(float a, float b, float *lo) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  *lo = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
  return s;
}

// x (two parts) + y * r (two parts each) + x.x * m, rounded once: the two
// halves of the addition theorem, with m = cos r - 1.
__device__ __forceinline__ float turn_by(float2 x, float2 y, float rh, float rl, float m) {
  const float p = __fmul_rn(y.x, rh);
  float e = __fmaf_rn(y.x, rh, -p);
  e = __fmaf_rn(y.x, rl, e);
  e = __fmaf_rn(y.y, rh, e);
  e = __fmaf_rn(x.x, m, e) + x.y;
  float lo;
  const float s = two_sum(x.x, p, &lo);
  return __fadd_rn(s, __fadd_rn(lo, e));
}

// table: kSin256, or a copy of it in shared memory (where many angles are taken: lanes
// read different entries).
__device__ __forceinline__ void rope_cos_sin_exact(int64_t rel, uint64_t phase, float *c, float *s,
                                                   const float2 *table = kSin256) {
  const uint64_t turns = static_cast<uint64_t>(rel) * phase;  // mod 2^64
  const uint64_t near = turns + (1ull << 55);
  const int k = static_cast<int>(near >> 56);  // the nearest 256th, 0 .. 255
  const int64_t rest = static_cast<int64_t>(near & ((1ull << 56) - 1)) - (1ll << 55);
  // sin and cos of k 256ths from the first quarter
  const int q = k >> 6, j = k & 63;
  float2 a = table[j], b = table[64 - j];  // sin, cos of j
  float2 sn = (q & 1) ? b : a, cs = (q & 1) ? a : b;
  if (q & 2) sn = make_float2(-sn.x, -sn.y);
  if (q == 1 || q == 2) cs = make_float2(-cs.x, -cs.y);
  // the rest in radians, two parts (its own two parts: 55 bits do not fit one)
  const float nh = static_cast<float>(rest);
  const float nl = static_cast<float>(rest - static_cast<int64_t>(nh));
  const float rh = __fmul_rn(nh, kTurnHi);
  float rl = __fmaf_rn(nh, kTurnHi, -rh);
  rl = __fmaf_rn(nh, kTurnLo, rl);
  rl = __fmaf_rn(nl, kTurnHi, rl);
  // sin r = r - r^3 / 6 + r^5 / 120, cos r - 1 = -r^2 / 2 + r^4 / 24: what is left out is
  // below 2^-53 (r^7 / 5040) and 2^-47 (r^6 / 720)
  const float r2 = __fmul_rn(rh, rh);
  const float sl = __fmaf_rn(rh * r2, __fmaf_rn(r2, 1.f / 120.f, -1.f / 6.f), rl);
  const float m = __fmaf_rn(r2, __fmaf_rn(r2, 1.f / 24.f, -0.5f), -rh * rl);
  *c = turn_by(cs, make_float2(-sn.x, -sn.y), rh, sl, m);
  *s = turn_by(sn, cs, rh, sl, m);
}

}  // namespace hw
