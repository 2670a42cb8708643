// hw_fp4.cuh - the 4-bit cache format (HW_FP4_E2M1), written and read.
//
// A token's key (or value) of one kv head is 128 E2M1 codes, two to a byte with the
// even element in the low bits, and one bf16 scale s = bf16(max|x| / 6); an element
// stands for level(code) * s with the levels 0, 1/2, 1, 3/2, 2, 3, 4, 6 and a sign.
// E2M1 is what the tensor cores take as an operand, so a tile goes from memory into
// the product without being widened, and a scale a token is one factor of a
// row of scores (keys) or of a weight (values).
// Codes are the nearest level to x / s, ties to the even code, of the exact quotient.
// A scale below 2^-100 counts as zero (and the codes with it); a token with an element of
// 2^100 or more, or not finite, gets the scale NaN: it reads as NaN.  (The attention kernel
// takes scales into exponents and back: this keeps both in range.)
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <stdint.h>

namespace hw {

// The scale of a token whose largest magnitude is `top` (NaN if one is NaN).
__device__ __forceinline__ float fp4_scale(float top) {
  const float s = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(top, 6.f)));
  if (!(top < 0x1p100f)) return __int_as_float(0x7fc00000);
  return s < 0x1p-100f ? 0.f : s;
}

// |x| and the running maximum, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

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

// The codes of 8 numbers under the scale s > 0, with inv = 1 / s.  The product with inv
// is off by less than 2^-22, so where 2^-20 to either side gives the same codes
// they are the quotient's; elsewhere (one word in ten thousand) borders decide.
__device__ __forceinline__ uint32_t fp4_encode8(const float (&x)[8], float s, float inv) {
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = x[i] * inv;
    lo[i] = t * (1.f - 0x1p-20f);
    hi[i] = t * (1.f + 0x1p-20f);
  }
  uint32_t w = e2m1x8(lo);
  if (w != e2m1x8(hi)) {
    w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= fp4_code_exact(x[i], s) << (4 * i);
  }
  return w;
}

// The same of 2 numbers.
__device__ __forceinline__ uint32_t fp4_encode2(float x, float y, float s, float inv) {
  const float tx = x * inv, ty = y * inv;
  uint32_t lo, hi;
  asm("{\n\t.reg .b8 a, b;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %3, %2;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %5, %4;\n\t"
      "mov.b32 %0, {a, a, a, a};\n\tmov.b32 %1, {b, b, b, b};\n\t}"
      : "=r"(lo), "=r"(hi)
      : "f"(tx * (1.f - 0x1p-20f)), "f"(ty * (1.f - 0x1p-20f)), "f"(tx * (1.f + 0x1p-20f)), "f"(ty * (1.f + 0x1p-20f)));
  if (lo != hi) return fp4_code_exact(x, s) | fp4_code_exact(y, s) << 4;
  return lo & 0xffu;
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
__device__ __forceinline__ float fp4_row(const float (&lo)[8], const float (&hi)[8], uint32_t &wlo, uint32_t &whi) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max_nan(top, max_nan(fabsf(lo[i]), fabsf(hi[i])));
  const float s = fp4_scale(max_of_8(top));
  wlo = whi = 0;
  if (s > 0.f) {
    const float inv = 1.f / s;
    wlo = fp4_encode8(lo, s, inv);
    whi = fp4_encode8(hi, s, inv);
  }
  return s;
}

// The pair (x0, x1) turned by the angle of (cos, sin).  Every product is rounded:
// what the codes become does not hang on how they are fused.
__device__ __forceinline__ void fp4_turn(float x0, float x1, float c, float s, float &y0, float &y1) {
  y0 = __fsub_rn(__fmul_rn(x0, c), __fmul_rn(x1, s));
  y1 = __fadd_rn(__fmul_rn(x1, c), __fmul_rn(x0, s));
}

// The two scales of a token as its word of kv_scale: the key's in the low half.
__device__ __forceinline__ uint32_t fp4_scale_word(float ks, float vs) {
  return __float_as_uint(ks) >> 16 | (__float_as_uint(vs) & 0xffff0000u);
}
__device__ __forceinline__ float fp4_k_scale(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float fp4_v_scale(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

}  // namespace hw
