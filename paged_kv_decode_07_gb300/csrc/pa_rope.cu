// pa_rope.cu -- position rotation and optional per-head RMS norm of the new
// tokens' queries and keys, and the quantised write of their keys and values
// into the paged cache, in one pass over the projection's output.
//
// Per (token, head) row x of D values, in fp32:
//   norm     x_d <- x_d * w_d / sqrt(mean(x^2) + eps)             (optional)
//   rotation pair i < rot / 2, angle a = position * inv_freq_i:
//            (x, y) <- f * (x cos a - y sin a, x sin a + y cos a),
//            the pair being (i, i + rot / 2) or (2 i, 2 i + 1)
// and one rounding at the end: bf16 for the queries, the cache's format for
// keys and values (the codes are those of the fp32 row, not of a bf16 one).
//
// Angles: position * inv_freq in fp32 is off by up to position * 2^-25
// radians (0.03 at 10^6), far more than a bf16 output shows, so the angle is
// kept in turns as a 64-bit fixed-point fraction: inv_freq / 2 pi is formed
// once per thread from the float's 24-bit integer (exact to 2^-62 relative),
// and the product with the position wraps modulo one turn by itself.  The
// top 32 bits go to sincospi.  fp64 would do as well, at this GPU's fp64 rate
// a few hundred cycles per warp.
//
// Layout: D / 16 lanes hold a row, each the two 8-element chunks that rotate
// with each other (half pairs) or any two chunks (interleaved pairs), so a
// pair never leaves a thread, every access is 16 bytes, and a lane's eight
// sines and cosines serve every head of its token.  rot is a multiple of 32,
// so the 16-element scale blocks of NVFP4 sit in neighbouring lanes.
//
// Bound by HBM, reads and writes mixed: 8,191 tokens of 24 + 4 heads of 256 with
// norms (268 MB) in 47.0 us, 5.7 TB/s or 0.84 of a pure copy; 32,768 tokens into an
// FP8 cache (1.0 GB) in 178 us, 0.83.
#include "pa_codec.cuh"
#include "pa_launch.h"

namespace pa {
namespace {

using namespace codec;

// one warp per CTA: a warp's slot is refilled as soon as it ends (28 per SM; with
// four warps a CTA 8191 tokens took 53 us instead of 48)
constexpr int kRopeCtas = 28;

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

// the row's codes (and scales) into the pool; every lane of the warp calls it
template <int DT, int D>
__device__ __forceinline__ void encode_row(const KvView &kv, int which, size_t row, int ca, int cb,
                                           const Pair16 &x, bool live) {
  constexpr int L = D / 16;
  void *data = const_cast<void *>(which ? kv.v : kv.k);
  void *scale = const_cast<void *>(which ? kv.vs : kv.ks);
  const float g = which ? kv.vg : kv.kg;
  if constexpr (DT == PA_KV_BF16) {
    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(data) + row * D * 2);
    if (live) {
      dst[ca] = pack8(x.a);
      dst[cb] = pack8(x.b);
    }
  } else if constexpr (DT == PA_KV_FP8) {
    uint2 *dst = reinterpret_cast<uint2 *>(static_cast<uint8_t *>(data) + row * D);
    if (live) {
      dst[ca] = fp8_codes8(x.a, g);
      dst[cb] = fp8_codes8(x.b, g);
    }
  } else if constexpr (DT == PA_KV_INT8) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fmaxf(fabsf(x.a[i]), fabsf(x.b[i])));
#pragma unroll
    for (int o = L / 2; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const __half s16 = int8_scale(amax);
    const float s = __half2float(s16);
    uint2 *dst = reinterpret_cast<uint2 *>(static_cast<uint8_t *>(data) + row * D);
    if (live) {
      dst[ca] = int8_codes8(x.a, s);
      dst[cb] = int8_codes8(x.b, s);
      if (threadIdx.x % L == 0) static_cast<__half *>(scale)[row] = s16;
    }
  } else {   // NVFP4: chunks 2m, 2m + 1 of a scale block are in neighbouring lanes
    float ma = 0.f, mb = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      ma = fmaxf(ma, fabsf(x.a[i]));
      mb = fmaxf(mb, fabsf(x.b[i]));
    }
    ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, 1));
    mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
    const uint32_t sa = nvfp4_scale(ma, g), sb = nvfp4_scale(mb, g);
    uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(data) + row * (D / 2));
    uint8_t *sdst = static_cast<uint8_t *>(scale) + row * (D / 16);
    if (live) {
      dst[ca] = nvfp4_codes8(x.a, sa, g);
      dst[cb] = nvfp4_codes8(x.b, sb, g);
      if (!(ca & 1)) sdst[ca >> 1] = (uint8_t)sa;
      if (!(cb & 1)) sdst[cb >> 1] = (uint8_t)sb;
    }
  }
}

// A token's rows are taken in steps of 32 / L heads of one kind: first the
// queries, then the keys, then the values.  One warp takes a run of a token's
// steps, the next one's rows (or two's) on their way while it is at one.
template <int DT, int D, bool IL>
__global__ void __launch_bounds__(32, kRopeCtas) rope_kernel(const RopeParams p) {
  constexpr int L = D / 16, RPW = 32 / L;
  const int lane = threadIdx.x, sub = lane / L, j = lane % L;
  const int t = blockIdx.x / p.parts, part = blockIdx.x % p.parts;
  const int Hq = p.Hq, Hkv = p.kv.hkv;
  const int sq = (Hq + RPW - 1) / RPW, skv = (Hkv + RPW - 1) / RPW;
  const int s0 = part * p.steps_per_part, s1 = min(sq + 2 * skv, s0 + p.steps_per_part);

  // this lane's two chunks
  const int nr = p.rot / 16;   // chunks per half of the rotated part
  int ca, cb;
  bool ra, rb;
  if constexpr (IL) {
    ca = j;
    cb = j + L;
    ra = ca * 8 < p.rot;
    rb = cb * 8 < p.rot;
  } else {
    ra = rb = j < nr;
    ca = ra ? j : nr + j;        // past the rotated part: 2 nr + (j - nr)
    cb = ra ? j + nr : ca + (L - nr);
  }
  // one step: its kind (uniform in the warp), this lane's head and chunks
  struct Step {
    int kind, h;
    bool live;
    uint4 a, b;
  };
  auto load = [&](int s) {
    Step x;
    x.kind = s < sq ? 0 : s < sq + skv ? 1 : 2;
    x.h = (x.kind == 0 ? s : x.kind == 1 ? s - sq : s - sq - skv) * RPW + sub;
    x.live = s < s1 && x.h < (x.kind == 0 ? Hq : Hkv);
    x.a = x.b = make_uint4(0, 0, 0, 0);
    if (x.live) {
      const __nv_bfloat16 *src = x.kind == 0   ? p.q + (size_t)t * p.q_stride
                                 : x.kind == 1 ? p.k + (size_t)t * p.k_stride
                                               : p.v + (size_t)t * p.v_stride;
      const uint4 *s4 = reinterpret_cast<const uint4 *>(src + (size_t)x.h * D);
      x.a = __ldg(s4 + ca);
      x.b = __ldg(s4 + cb);
    }
    return x;
  };
  // bf16 caches, D = 256: two steps' rows on their way (8,191 tokens 48.3 -> 47.0 us,
  // 32,768 173 -> 165).  The others have no registers for it (FP8 178 -> 266 us) or
  // half the steps (D = 128: 49.2 -> 50.0 us).
  constexpr bool TWO = DT == PA_KV_BF16 && D == 256;
  Step x0 = load(s0), x1;
  if constexpr (TWO) x1 = load(s0 + 1);
  // the angles of this lane's pairs, once for every head of the token
  float cs[8], sn[8];
  const int pos = __ldg(p.positions + t);
  const int64_t slot = __ldg(p.slots + t);
  if ((ra || rb) && s0 < sq + skv) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int pair = IL ? (i < 4 ? 4 * ca + i : 4 * cb + i - 4) : 8 * j + i;
      cs[i] = pair < p.rot / 2 ? __ldg(p.inv_freq + pair) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t ph = turns_per_position(cs[i]) * (uint64_t)(int64_t)pos;
      // half turns in [-1, 1): the top 32 bits of the phase, as a signed number
      sincospif((float)(int32_t)(uint32_t)(ph >> 32) * 0x1p-31f, &sn[i], &cs[i]);
      cs[i] *= p.factor;
      sn[i] *= p.factor;
    }
  }
  const int64_t nslots = (int64_t)p.kv.num_blocks * kBlock;
  const bool bad = slot < -1 || slot >= nslots;
  if (bad && part == 0 && lane == 0) set_err(p.hdr, PA_ERRF_BAD_SLOT);
  const bool keep = slot >= 0 && !bad;
  const size_t row0 = keep ? (size_t)(slot >> 4) * Hkv * kBlock + (size_t)(slot & 15) : 0;

  auto finish = [&](const Step &st) {
    Pair16 x;
    unpack8(st.a, x.a);
    unpack8(st.b, x.b);
    const __nv_bfloat16 *const w = st.kind == 0 ? p.q_norm : st.kind == 1 ? p.k_norm : nullptr;
    if (w) {
      const uint4 *w4 = reinterpret_cast<const uint4 *>(w);
      rms_norm<D>(x, __ldg(w4 + ca), __ldg(w4 + cb), p.eps);
    }
    if (st.kind < 2) rotate<IL>(x, cs, sn, ra, rb);
    if (st.kind == 0) {
      if (st.live) {
        uint4 *dst = reinterpret_cast<uint4 *>(p.q_out + (size_t)t * p.q_out_stride + (size_t)st.h * D);
        dst[ca] = pack8(x.a);
        dst[cb] = pack8(x.b);
      }
      return;
    }
    encode_row<DT, D>(p.kv, st.kind == 2, row0 + (size_t)st.h * kBlock, ca, cb, x, st.live && keep);
  };
#pragma unroll 1
  for (int s = s0; s < s1; s += TWO ? 2 : 1) {
    const Step y = x0;
    if constexpr (TWO)
      x0 = load(s + 2);
    else if (s + 1 < s1)
      x0 = load(s + 1);
    finish(y);
    if constexpr (TWO) {
      if (s + 1 < s1) {
        const Step z = x1;
        x1 = load(s + 3);
        finish(z);
      }
    }
  }
}

template <int DT, int D>
cudaError_t launch_dt(const RopeParams &p, unsigned grid, cudaStream_t s) {
  if (p.interleaved)
    rope_kernel<DT, D, true><<<grid, 32, 0, s>>>(p);
  else
    rope_kernel<DT, D, false><<<grid, 32, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(RopeParams p, cudaStream_t s) {
  const int rpw = 512 / p.kv.D;   // heads a step takes
  const int steps = (p.Hq + rpw - 1) / rpw + 2 * ((p.kv.hkv + rpw - 1) / rpw);
  // few tokens: a token's steps are spread over several warps, about
  // sixteen warps per SM in all (255 tokens: 6.0 us, with eight 7.0, with 56 6.5)
  const int want = (2432 + p.T - 1) / p.T;
  const int parts = want < 1 ? 1 : want > steps ? steps : want;
  p.steps_per_part = (steps + parts - 1) / parts;
  p.parts = (steps + p.steps_per_part - 1) / p.steps_per_part;
  const unsigned grid = (unsigned)p.T * (unsigned)p.parts;   // below 2^30 (rows are)
  switch (p.kv.dtype * 2 + (p.kv.D == 256)) {
    case PA_KV_BF16 * 2: return launch_dt<PA_KV_BF16, 128>(p, grid, s);
    case PA_KV_BF16 * 2 + 1: return launch_dt<PA_KV_BF16, 256>(p, grid, s);
    case PA_KV_INT8 * 2: return launch_dt<PA_KV_INT8, 128>(p, grid, s);
    case PA_KV_INT8 * 2 + 1: return launch_dt<PA_KV_INT8, 256>(p, grid, s);
    case PA_KV_NVFP4 * 2: return launch_dt<PA_KV_NVFP4, 128>(p, grid, s);
    case PA_KV_NVFP4 * 2 + 1: return launch_dt<PA_KV_NVFP4, 256>(p, grid, s);
    case PA_KV_FP8 * 2: return launch_dt<PA_KV_FP8, 128>(p, grid, s);
    case PA_KV_FP8 * 2 + 1: return launch_dt<PA_KV_FP8, 256>(p, grid, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace pa
