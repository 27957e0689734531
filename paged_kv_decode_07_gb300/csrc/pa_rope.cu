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
#include "pa_codec.cuh"
#include "pa_launch.h"

namespace pa {
namespace {

using namespace codec;

constexpr int kRopeWarps = 4;

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

// norm, rotate and round 16 values of a row held by a lane (two chunks)
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
  float s0 = 0.f, s1 = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    s0 = fmaf(x.a[i], x.a[i], s0);
    s1 = fmaf(x.b[i], x.b[i], s1);
  }
  float s = s0 + s1;
#pragma unroll
  for (int o = L / 2; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const float r = rsqrtf(s * (1.0f / D) + eps);
  float w[8];
  unpack8(wa, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) x.a[i] = x.a[i] * r * w[i];
  unpack8(wb, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) x.b[i] = x.b[i] * r * w[i];
}

template <bool IL>
__device__ __forceinline__ void rotate(Pair16 &x, const float (&cs)[8], const float (&sn)[8],
                                       bool ra, bool rb) {
  if constexpr (IL) {   // pairs inside each chunk
    if (ra) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float u = x.a[2 * i], v = x.a[2 * i + 1];
        x.a[2 * i] = u * cs[i] - v * sn[i];
        x.a[2 * i + 1] = u * sn[i] + v * cs[i];
      }
    }
    if (rb) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float u = x.b[2 * i], v = x.b[2 * i + 1];
        x.b[2 * i] = u * cs[4 + i] - v * sn[4 + i];
        x.b[2 * i + 1] = u * sn[4 + i] + v * cs[4 + i];
      }
    }
  } else if (ra) {      // element i of the first chunk with element i of the second
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float u = x.a[i], v = x.b[i];
      x.a[i] = u * cs[i] - v * sn[i];
      x.b[i] = u * sn[i] + v * cs[i];
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

// One warp takes rows [part * per, ...) of a token's Hq + 2 Hkv rows (q
// heads, then k, then v); 32 / L rows at a time.
template <int DT, int D, bool IL>
__global__ void __launch_bounds__(kRopeWarps * 32) rope_kernel(const RopeParams p) {
  constexpr int L = D / 16, RPW = 32 / L;
  const int lane = threadIdx.x & 31, sub = lane / L, j = lane % L;
  const long long w = (long long)blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
  const int t = (int)(w / p.parts), part = (int)(w % p.parts);
  if (t >= p.T) return;
  const int Hq = p.Hq, Hkv = p.kv.hkv;
  const int rows = Hq + 2 * Hkv;
  const int r_end = min(rows, (part + 1) * p.rows_per_part);

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
  // the angles of this lane's pairs, once for every head of the token
  float cs[8], sn[8];
  const int pos = __ldg(p.positions + t);
  if (ra || rb) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int pair = IL ? (i < 4 ? 4 * ca + i : 4 * cb + i - 4) : 8 * j + i;
      float c = 1.f, s = 0.f;
      if (pair < p.rot / 2) {
        const uint64_t ph = turns_per_position(__ldg(p.inv_freq + pair)) * (uint64_t)(int64_t)pos;
        // half turns in [-1, 1): the top 32 bits of the phase, as a signed number
        sincospif((float)(int32_t)(uint32_t)(ph >> 32) * 0x1p-31f, &s, &c);
      }
      cs[i] = c * p.factor;
      sn[i] = s * p.factor;
    }
  }
  const int64_t slot = __ldg(p.slots + t);
  const int64_t nslots = (int64_t)p.kv.num_blocks * kBlock;
  const bool bad = slot < -1 || slot >= nslots;
  if (bad && part == 0 && lane == 0) set_err(p.hdr, PA_ERRF_BAD_SLOT);
  const bool keep = slot >= 0 && !bad;

  for (int r0 = part * p.rows_per_part; r0 < r_end; r0 += RPW) {
    const int r = r0 + sub;
    const bool live = r < r_end;
    const int kind = r < Hq ? 0 : r < Hq + Hkv ? 1 : 2;
    const int h = kind == 0 ? r : kind == 1 ? r - Hq : r - Hq - Hkv;
    const __nv_bfloat16 *src = kind == 0   ? p.q + (size_t)t * p.q_stride
                               : kind == 1 ? p.k + (size_t)t * p.k_stride
                                           : p.v + (size_t)t * p.v_stride;
    Pair16 x;
    if (live) {
      const uint4 *s4 = reinterpret_cast<const uint4 *>(src + (size_t)h * D);
      unpack8(__ldcs(s4 + ca), x.a);
      unpack8(__ldcs(s4 + cb), x.b);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x.a[i] = x.b[i] = 0.f;
    }
    if (p.q_norm || p.k_norm) {
      Pair16 y = x;
      const __nv_bfloat16 *w = kind == 0 ? p.q_norm : p.k_norm;
      uint4 wa = make_uint4(0, 0, 0, 0), wb = wa;
      if (w) {
        wa = __ldg(reinterpret_cast<const uint4 *>(w) + ca);
        wb = __ldg(reinterpret_cast<const uint4 *>(w) + cb);
      }
      rms_norm<D>(y, wa, wb, p.eps);
      if (kind < 2 && w) x = y;
    }
    if (kind < 2) rotate<IL>(x, cs, sn, ra, rb);
    if (kind == 0 && live) {
      uint4 *dst = reinterpret_cast<uint4 *>(p.q_out + (size_t)t * p.q_out_stride + (size_t)h * D);
      dst[ca] = pack8(x.a);
      dst[cb] = pack8(x.b);
    }
    if (__any_sync(0xffffffffu, kind > 0)) {
      const size_t row = keep ? ((size_t)(slot >> 4) * Hkv + h) * kBlock + (size_t)(slot & 15) : 0;
      encode_row<DT, D>(p.kv, kind == 2, row, ca, cb, x, live && kind > 0 && keep);
    }
  }
}

template <int DT, int D>
cudaError_t launch_dt(const RopeParams &p, unsigned grid, cudaStream_t s) {
  if (p.interleaved)
    rope_kernel<DT, D, true><<<grid, kRopeWarps * 32, 0, s>>>(p);
  else
    rope_kernel<DT, D, false><<<grid, kRopeWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(RopeParams p, cudaStream_t s) {
  const int rpw = 512 / p.kv.D;   // rows a warp takes at a time
  const int rows = p.Hq + 2 * p.kv.hkv;
  p.parts = 1;
  p.rows_per_part = (rows + rpw - 1) / rpw * rpw;
  const long long warps = (long long)p.T * p.parts;
  const unsigned grid = (unsigned)((warps + kRopeWarps - 1) / kRopeWarps);
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
