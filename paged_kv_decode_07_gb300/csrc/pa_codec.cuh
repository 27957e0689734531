// pa_codec.cuh -- encoding of fp32 values into the quantised KV formats
// (round to nearest even, saturating), shared by the kernels that write the
// cache.  Every rounding decision is that of the IEEE fp32 quotient.
#pragma once

#include "pa_internal.cuh"

namespace pa {
namespace codec {

// (lo, hi) -> two E4M3 codes, lo in the low byte; round to nearest even,
// saturating at 448
__device__ __forceinline__ uint32_t e4m3x2_rn_sat(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// eight magnitudes -> eight E2M1 codes, element 2i in the low nibble of byte i
__device__ __forceinline__ uint32_t e2m1x8_rn_sat(const float (&a)[8]) {
  uint32_t r;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      " mov.b32 %0, {b0, b1, b2, b3};\n}\n"
      : "=r"(r)
      : "f"(a[0]), "f"(a[1]), "f"(a[2]), "f"(a[3]), "f"(a[4]), "f"(a[5]), "f"(a[6]), "f"(a[7]));
  return r;
}

__device__ __forceinline__ float e4m3_to_float(uint32_t code) {
  return __half2float(__ushort_as_half((uint16_t)(e4m3x2_u16_to_h2(code) & 0xFFFFu)));
}

// ---- quotients without a division per element.  With r an approximate
// reciprocal of the divisor d (rcp.approx, at most 1 ulp off, i.e. a
// relative error below 2^-23), RN(x * r) lies within 2^-22 of the IEEE
// quotient RN(x / d), relatively.  Rounding onto a grid (integers, fp16,
// E4M3, E2M1) is monotone, so the decision is taken at both ends of a
// bracket that must hold the exact quotient -- x * RN(r * (1 -+ 2^-20)) --
// and when the two ends agree that is the decision of RN(x / d) itself.
// Otherwise (a few in 10^5 elements) the quotient is formed exactly.  For
// int8 the bracket is the distance to the nearest half integer instead:
// |x / d| < 2^8 there, so RN(x * r) is within 2^-14 of RN(x / d) and a
// margin of 2^-13 decides.
constexpr float kBracketLo = 1.0f - 0x1p-20f;
constexpr float kBracketHi = 1.0f + 0x1p-20f;
constexpr float kInf = __builtin_huge_valf();

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(*reinterpret_cast<unsigned long long *>(&d))
      : "l"(*reinterpret_cast<unsigned long long *>(&a)),
        "l"(*reinterpret_cast<unsigned long long *>(&b)));
  return d;
}

__device__ __forceinline__ float2 fsub2(float2 a, float2 b) {
  float2 d;
  asm("sub.rn.f32x2 %0, %1, %2;"
      : "=l"(*reinterpret_cast<unsigned long long *>(&d))
      : "l"(*reinterpret_cast<unsigned long long *>(&a)),
        "l"(*reinterpret_cast<unsigned long long *>(&b)));
  return d;
}

// low bytes of four words -> one word
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040u), __byte_perm(c, d, 0x0040u), 0x5410u);
}

// E4M3 codes of RN(x / d) for EPL values, 4 per word; `ok` = false when the
// bracket could not decide (the caller then forms exact quotients)
template <int EPL>
__device__ __forceinline__ void e4m3_codes(const float (&x)[EPL], float rlo, float rhi,
                                           uint32_t (&w)[EPL / 4], bool &ok) {
#pragma unroll
  for (int k = 0; k < EPL / 4; ++k) {
    const float2 a = fmul2(make_float2(x[4 * k], x[4 * k + 1]), make_float2(rlo, rlo));
    const float2 b = fmul2(make_float2(x[4 * k + 2], x[4 * k + 3]), make_float2(rlo, rlo));
    const float2 c = fmul2(make_float2(x[4 * k], x[4 * k + 1]), make_float2(rhi, rhi));
    const float2 e = fmul2(make_float2(x[4 * k + 2], x[4 * k + 3]), make_float2(rhi, rhi));
    const uint32_t lo = __byte_perm(e4m3x2_rn_sat(a.x, a.y), e4m3x2_rn_sat(b.x, b.y), 0x5410u);
    const uint32_t hi = __byte_perm(e4m3x2_rn_sat(c.x, c.y), e4m3x2_rn_sat(e.x, e.y), 0x5410u);
    ok = ok && lo == hi;
    w[k] = lo;
  }
}

// a byte whose magnitude bits are 0 is written +0
__device__ __forceinline__ uint32_t plus_zero(uint32_t w) {
  const uint32_t nz = (w & 0x7F7F7F7Fu) + 0x7F7F7F7Fu;   // bit 7 set iff magnitude != 0
  return w & (nz | 0x7F7F7F7Fu);
}

// ---- whole 8-value pieces of a row (two code words, 4 one-byte codes each,
// or one word of 8 nibbles)

// fp16 scale of an int8 row: fp16_RN(RN(amax / 127))
__device__ __forceinline__ __half int8_scale(float amax) {
  constexpr float r127 = 1.0f / 127.0f;
  const __half s = __float2half_rn(__fmul_rn(amax, r127 * kBracketLo));
  if (__half_as_ushort(s) == __half_as_ushort(__float2half_rn(__fmul_rn(amax, r127 * kBracketHi))))
    return s;
  return __float2half_rn(__fdiv_rn(amax, 127.0f));
}

// int8 codes of x / s (s > 0, else zeros): the quotient's distance to the
// nearest half integer decides whether the approximate one may be rounded
__device__ __forceinline__ uint2 int8_codes8(const float (&x)[8], float s) {
  if (!(s > 0.f)) return make_uint2(0, 0);
  const float rs = rcp_approx(s);
  constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: adding it rounds to an integer (RNE)
  bool near = false;
  float t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = fminf(fmaxf(x[i] * rs, -127.f), 127.f);   // subnormal s: |x / s| may pass 127.5
    const float tt = q + kMagic;
    near = near || fabsf(q - (tt - kMagic)) > 0.5f - 0x1p-13f;
    t[i] = tt;
  }
  if (near) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      t[i] = __uint_as_float((uint32_t)max(-127, min(127, __float2int_rn(__fdiv_rn(x[i], s)))));
  }
  return make_uint2(low_bytes(__float_as_uint(t[0]), __float_as_uint(t[1]), __float_as_uint(t[2]),
                              __float_as_uint(t[3])),
                    low_bytes(__float_as_uint(t[4]), __float_as_uint(t[5]), __float_as_uint(t[6]),
                              __float_as_uint(t[7])));
}

// E4M3 codes of x / g with the zero magnitude written +0 (g <= 0: zeros)
__device__ __forceinline__ uint2 fp8_codes8(const float (&x)[8], float g) {
  const float rg = rcp_approx(g);
  bool ok = g > 0.f && rg < kInf;
  uint32_t w[2];
  e4m3_codes<8>(x, __fmul_rn(rg, kBracketLo), __fmul_rn(rg, kBracketHi), w, ok);
  if (!ok) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = g > 0.f ? __fdiv_rn(x[4 * k + j], g) : 0.f;
      w[k] = __byte_perm(e4m3x2_rn_sat(y[0], y[1]), e4m3x2_rn_sat(y[2], y[3]), 0x5410u);
    }
  }
  return make_uint2(plus_zero(w[0]), plus_zero(w[1]));
}

// E4M3 scale byte of a 16-element block: E4M3_RN(RN(amax / RN(g * 6)))
__device__ __forceinline__ uint32_t nvfp4_scale(float amax, float g) {
  const float den = __fmul_rn(g, 6.0f);
  const float rden = rcp_approx(den);
  const uint32_t lo = e4m3x2_rn_sat(__fmul_rn(amax, __fmul_rn(rden, kBracketLo)), 0.f) & 0xFFu;
  const uint32_t hi = e4m3x2_rn_sat(__fmul_rn(amax, __fmul_rn(rden, kBracketHi)), 0.f) & 0xFFu;
  if (g > 0.f && rden < kInf && lo == hi) return lo;
  return g > 0.f ? (e4m3x2_rn_sat(__fdiv_rn(amax, den), 0.f) & 0xFFu) : 0u;
}

// E2M1 codes of x / (e4m3(scale) * g), element 2i in the low nibble
__device__ __forceinline__ uint32_t nvfp4_codes8(const float (&x)[8], uint32_t scale, float g) {
  const float sg = __fmul_rn(e4m3_to_float(scale), g);
  if (!(sg > 0.f)) return 0u;   // the quotient is taken as +0
  const float r = rcp_approx(sg);
  const float rlo = __fmul_rn(r, kBracketLo), rhi = __fmul_rn(r, kBracketHi);
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo[i] = x[i] * rlo;
    hi[i] = x[i] * rhi;
  }
  uint32_t c = e2m1x8_rn_sat(lo);
  if (!(r < kInf) || c != e2m1x8_rn_sat(hi)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) lo[i] = __fdiv_rn(x[i], sg);
    c = e2m1x8_rn_sat(lo);
  }
  return c;
}

}  // namespace codec
}  // namespace pa
