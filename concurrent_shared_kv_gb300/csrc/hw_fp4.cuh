// hw_fp4.cuh - the 4-bit cache format (HW_FP4_E2M1), written and read.
//
// A token's key (or value) of one kv head is 128 E2M1 codes, two to a byte with the
// even element in the low bits, and one bf16 scale s = bf16(max|x| (1 / 6)); an element
// stands for level(code) * s with the levels 0, 1/2, 1, 3/2, 2, 3, 4, 6 and a sign.
// E2M1 is what the tensor cores take as an operand, so a tile goes from memory into
// the product without being widened, and a scale a token is one factor of a
// row of scores (keys) or of a weight (values).
// Codes are the nearest level to x / s, ties to the even code, of the exact quotient.  (Keys
// that a commit turns: of a quotient that is off by up to 2^-21, see commit_key.)
// A scale below 2^-100 counts as zero (and the codes with it); a token with an element of
// 2^100 or more, or not finite, gets the scale NaN: it reads as NaN.  (Products of scales, codes and
// weights then stay inside fp32's range.)
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <stdint.h>

namespace hw {

// The scale of a token whose largest magnitude is `top` (NaN if one is NaN).  (A sixth to
// 2^-23 beside a scale's 2^-8.)
__device__ __forceinline__ float fp4_scale(float top) {
  const float s = __bfloat162float(__float2bfloat16_rn(__fmul_rn(top, 1.f / 6.f)));
  if (!(top < 0x1p100f)) return __int_as_float(0x7fc00000);
  return s < 0x1p-100f ? 0.f : s;
}

// |x| and the running maximum, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
  return d;
}
__device__ __forceinline__ float2 fpair2(float x) { return make_float2(x, x); }

// The nearest codes of 8 numbers already in units of the scale, the first one lowest.
__device__ __forceinline__ uint32_t e2m1x8(const float (&t)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(t[0]), "f"(t[1]), "f"(t[2]), "f"(t[3]), "f"(t[4]), "f"(t[5]), "f"(t[6]), "f"(t[7]));
  return w;
}

// The nearest code of x under the scale s: borders between levels have at most
// 3 bits, a scale has 8, so their products are exact.
__device__ __forceinline__ uint32_t fp4_code_exact(float x, float s) {
  const float a = fabsf(x);
  uint32_t c = 0;
  c += a > 0.25f * s;
  c += a >= 0.75f * s;
  c += a > 1.25f * s;
  c += a >= 1.75f * s;
  c += a > 2.5f * s;
  c += a >= 3.5f * s;
  c += a > 5.f * s;
  return c | (__float_as_uint(x) >> 28 & 8u);
}

// The codes of 8 numbers under the scale s > 0.  A product with 1 / s is off by less than
// 2^-22, so where 2^-20 to either side give the same code it is the quotient's; at the few
// elements where they do not, the border between the two decides.
__device__ __forceinline__ uint32_t fp4_encode8(const float (&x)[8], float s) {
  const float inv = 1.f / s, inv_lo = inv * (1.f - 0x1p-20f), inv_hi = inv * (1.f + 0x1p-20f);
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 a = __fmul2_rn(make_float2(x[i], x[i + 1]), fpair2(inv_lo));
    const float2 b = __fmul2_rn(make_float2(x[i], x[i + 1]), fpair2(inv_hi));
    lo[i] = a.x;
    lo[i + 1] = a.y;
    hi[i] = b.x;
    hi[i + 1] = b.y;
  }
  uint32_t w = e2m1x8(lo);
  const uint32_t diff = w ^ e2m1x8(hi);
  if (diff) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (diff >> (4 * i) & 0xfu) w = (w & ~(0xfu << (4 * i))) | fp4_code_exact(x[i], s) << (4 * i);
  }
  return w;
}

// The same for numbers of bf16: a quotient then is a border or 2^-11 of one away (8 bits
// against 8 times 3), so that rounded to 14 bits it stands on the right side of it, or
// on it.  (Ties are common among such numbers.)
__device__ __forceinline__ float fp4_snap(float t) { return __uint_as_float((__float_as_uint(t) + 0x200u) & ~0x3ffu); }
__device__ __forceinline__ uint32_t fp4_encode8_bf16(const float (&x)[8], float s) {
  const float inv = 1.f / s;
  float t[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 a = __fmul2_rn(make_float2(x[i], x[i + 1]), fpair2(inv));
    t[i] = fp4_snap(a.x);
    t[i + 1] = fp4_snap(a.y);
  }
  return e2m1x8(t);
}

// Of 2 numbers.
__device__ __forceinline__ uint32_t e2m1x2(float x, float y) {
  uint32_t w;
  asm("{\n\t.reg .b8 a;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tmov.b32 %0, {a, a, a, a};\n\t}" : "=r"(w) : "f"(x), "f"(y));
  return w & 0xffu;
}
__device__ __forceinline__ uint32_t fp4_encode2(float x, float y, float s) {
  const float inv = 1.f / s, lo = inv * (1.f - 0x1p-20f), hi = inv * (1.f + 0x1p-20f);
  const uint32_t w = e2m1x2(x * lo, y * lo);
  return w == e2m1x2(x * hi, y * hi) ? w : fp4_code_exact(x, s) | fp4_code_exact(y, s) << 4;
}
__device__ __forceinline__ uint32_t fp4_encode2_bf16(float x, float y, float s) {
  const float inv = 1.f / s;
  return e2m1x2(fp4_snap(x * inv), fp4_snap(y * inv));
}

// The levels (with signs) of 8 codes.
__device__ __forceinline__ void fp4_levels8(uint32_t w, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h(__nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(w >> (8 * i) & 0xffu), __NV_E2M1));
    const float2 f = __half22float2(h);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// The larger of `top` over the 8 neighbouring threads that hold a row.
__device__ __forceinline__ float max_of_8(float top) {
#pragma unroll
  for (int o = 4; o >= 1; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  return top;
}

// A row of 128 elements among 8 threads, each with the 8 of `lo` (from 8c) and the 8
// of `hi` (from 64 + 8c): its scale, and the thread's codes.  Whole warps call it.
// kBf16: the elements are numbers of bf16.
template <bool kBf16>
__device__ __forceinline__ float fp4_row(const float (&lo)[8], const float (&hi)[8], uint32_t &wlo, uint32_t &whi) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max3_abs_nan(top, lo[i], hi[i]);
  const float s = fp4_scale(max_of_8(top));
  wlo = whi = 0;
  if (s > 0.f) {
    wlo = kBf16 ? fp4_encode8_bf16(lo, s) : fp4_encode8(lo, s);
    whi = kBf16 ? fp4_encode8_bf16(hi, s) : fp4_encode8(hi, s);
  }
  return s;
}

// The pair (x0, x1) turned by the angle of (cos, sin).  Every product is rounded:
// what the codes become does not hang on how they are fused.
__device__ __forceinline__ void fp4_turn(float x0, float x1, float c, float s, float &y0, float &y1) {
  y0 = __fsub_rn(__fmul_rn(x0, c), __fmul_rn(x1, s));
  y1 = __fadd_rn(__fmul_rn(x1, c), __fmul_rn(x0, s));
}

// Two neighbouring pairs at once.
__device__ __forceinline__ void fp4_turn2(float2 x0, float2 x1, float2 c, float2 s, float2 &y0, float2 &y1) {
  const float2 d = __fmul2_rn(x1, s);
  y0 = __fadd2_rn(__fmul2_rn(x0, c), make_float2(-d.x, -d.y));
  y1 = __fadd2_rn(__fmul2_rn(x1, c), __fmul2_rn(x0, s));
}

// The two scales of a token as its word of kv_scale: the key's in the low half.
__device__ __forceinline__ uint32_t fp4_scale_word(float ks, float vs) {
  return __float_as_uint(ks) >> 16 | (__float_as_uint(vs) & 0xffff0000u);
}
__device__ __forceinline__ float fp4_k_scale(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float fp4_v_scale(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

}  // namespace hw
