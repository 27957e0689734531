// pa_rotate.cuh -- position rotation of rows held sixteen values a lane, shared
// by the kernels that write the caches (the mathematics: pa_rope.cu).
#pragma once

#include "pa_internal.cuh"

namespace pa {
namespace rotary {

// inv_freq (radians per position) -> turns per position in units of 2^-64.
// f = m * 2^(e - 126) with m in [1/2, 1) held as 64 fraction bits; 1 / 2 pi as
// a 64-bit fraction.
__device__ __forceinline__ uint64_t turns_per_position(float f) {
  constexpr uint64_t kInv2Pi = 0x28BE60DB9391054Aull;   // floor(2^64 / (2 pi))
  const uint32_t u = __float_as_uint(fabsf(f));
  const int e = (int)(u >> 23);
  if (e == 0 || e == 255) return 0;   // below 2^-126, or not finite: no rotation
  const uint64_t m = (uint64_t)((u & 0x7FFFFFu) | 0x800000u) << 40;
  const uint64_t p = __umul64hi(m, kInv2Pi);
  const int sh = 126 - e;
  const uint64_t t = sh >= 64 ? 0 : sh >= 0 ? p >> sh : -sh >= 64 ? 0 : p << -sh;
  return f < 0.f ? 0 - t : t;
}

// the 16 values of a row that a lane holds (two chunks of 8)
struct Pair16 {
  float a[8], b[8];
};

__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = bf16x2_to_f2(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]), pack_bf2(x[4], x[5]),
                    pack_bf2(x[6], x[7]));
}

// x * w / rms over the row's L lanes
template <int D>
__device__ __forceinline__ void rms_norm(Pair16 &x, const uint4 &wa, const uint4 &wb, float eps) {
  constexpr int L = D / 16;
  float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 a = make_float2(x.a[i], x.a[i + 1]), b = make_float2(x.b[i], x.b[i + 1]);
    s0 = ffma2(a, a, s0);
    s1 = ffma2(b, b, s1);
  }
  float s = (s0.x + s0.y) + (s1.x + s1.y);
#pragma unroll
  for (int o = L / 2; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const float r = rsqrtf(s * (1.0f / D) + eps);
  const float2 rr = make_float2(r, r);
  const uint32_t ua[4] = {wa.x, wa.y, wa.z, wa.w}, ub[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = fmul2(fmul2(make_float2(x.a[2 * i], x.a[2 * i + 1]), rr), bf16x2_to_f2(ua[i]));
    const float2 z = fmul2(fmul2(make_float2(x.b[2 * i], x.b[2 * i + 1]), rr), bf16x2_to_f2(ub[i]));
    x.a[2 * i] = y.x;
    x.a[2 * i + 1] = y.y;
    x.b[2 * i] = z.x;
    x.b[2 * i + 1] = z.y;
  }
}

// (x, y) <- (x c - y s, x s + y c) for every pair of the lane; cs, sn hold the
// pairs' cosines and sines (times the factor)
template <bool IL>
__device__ __forceinline__ void rotate(Pair16 &x, const float (&cs)[8], const float (&sn)[8],
                                       bool ra, bool rb) {
  auto inside = [&](float (&v)[8], int k) {   // pairs (2 i, 2 i + 1) of one chunk
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = ffma2(make_float2(v[2 * i + 1], v[2 * i + 1]), make_float2(-sn[k + i], cs[k + i]),
                             fmul2(make_float2(v[2 * i], v[2 * i]), make_float2(cs[k + i], sn[k + i])));
      v[2 * i] = y.x;
      v[2 * i + 1] = y.y;
    }
  };
  if constexpr (IL) {
    if (ra) inside(x.a, 0);
    if (rb) inside(x.b, 4);
  } else if (ra) {      // element i of the first chunk with element i of the second
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 u = make_float2(x.a[i], x.a[i + 1]), v = make_float2(x.b[i], x.b[i + 1]);
      const float2 c = make_float2(cs[i], cs[i + 1]), t = make_float2(sn[i], sn[i + 1]);
      const float2 y = ffma2(make_float2(-v.x, -v.y), t, fmul2(u, c));
      const float2 z = ffma2(v, c, fmul2(u, t));
      x.a[i] = y.x;
      x.a[i + 1] = y.y;
      x.b[i] = z.x;
      x.b[i + 1] = z.y;
    }
  }
}

// cosine and sine (times `factor`) of position * inv_freq: half turns in
// [-1, 1), the top 32 bits of the phase as a signed number
__device__ __forceinline__ void angle(float inv_freq, int pos, float factor, float &c, float &s) {
  const uint64_t ph = turns_per_position(inv_freq) * (uint64_t)(int64_t)pos;
  sincospif((float)(int32_t)(uint32_t)(ph >> 32) * 0x1p-31f, &s, &c);
  c *= factor;
  s *= factor;
}

}  // namespace rotary
}  // namespace pa
