// pa_score.cuh -- score options shared by the prefill and the scored decode
// kernels: tanh cap, distance bias, sliding window, first visible key and
// bidirectional prefix.
//
// Every mask here leaves a query one range [lo, hi) of keys, so a kernel
// skips the key tiles outside the range, masks the two ragged ends and
// treats the tiles between as dense.
#pragma once

#include "pa_internal.cuh"

namespace pa {

// keys [lo, hi) visible to the query at position pos of a sequence of n keys
struct KeyRange {
  int lo, hi;
};

__device__ __forceinline__ KeyRange key_range(const ScoreView &sc, int pos, int n, int first,
                                              int prefix) {
  KeyRange r;
  r.hi = min(n, max(pos + 1, prefix));
  r.lo = max(0, first);
  if (sc.window > 0) r.lo = max(r.lo, pos - sc.window + 1);
  if (pos < 0 || r.lo >= r.hi) r.lo = r.hi = 0;
  return r;
}

__device__ __forceinline__ float score_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float score_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// cap * tanh(s / cap) * log2 e from y = 2 log2 e * s / cap:
// tanh(u) = 1 - 2 / (1 + e^2u).  ex2 and rcp are good to about 2^-22, so the
// result is off by cap * 2^-21 at most (1e-5 of a probability at cap = 30);
// tanh.approx, at 2^-11, would be off by a hundredth of a score.
__device__ __forceinline__ float capped(float y, float cap_log2) {
  return fmaf(-2.f * cap_log2, score_rcp(1.f + score_ex2(y)), cap_log2);
}

// Under a cap above some 180 that error reaches 2^-13 of a score unit, so there
// scores below 0.4 cap come from a polynomial instead (see TanhSmall in
// pa_prefill_umma.cuh), whose error is relative to the score.
constexpr float kBigCap = 256.f;   // times log2 e
__device__ __forceinline__ float capped_big(float y, float cap_log2) {
  const float u = y * 0.34657359027997264f, v = u * u;
  if (fabsf(u) > 0.4f) return capped(y, cap_log2);
  const float h = fmaf(v, fmaf(v, fmaf(v, -0.0475493483f, 0.132708743f), -0.333313555f), 0.999999881f);
  return cap_log2 * (u * h);
}

}  // namespace pa
