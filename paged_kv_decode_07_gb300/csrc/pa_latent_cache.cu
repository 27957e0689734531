// pa_latent_cache.cu -- the latent cache's write (norm, rotation, rounding into
// slots) and its read-back as contiguous rows.
//
// Write, per token, in fp32 and rounded once at the end:
//   latent  c_d <- c_d * w_d / sqrt(mean(c^2) + eps)                 (optional)
//   rope    (x, y) <- f * (x cos a - y sin a, x sin a + y cos a), a = position *
//           inv_freq, of the token's 64 rotated values and of the 64 of every
//           head's query
// A warp takes a run of a token's steps: the latent (16 values a lane), or eight
// 64-value rows, four lanes each, a lane's two 8-value chunks holding whole
// pairs, so that eight sines and cosines serve every head.  Each lane computes one
// pair's and shuffles hand them out (eight a lane: 8,191 tokens 34.8 us, 31.4 so).
//
// Both kernels move bytes.  Many rows are bound by HBM: 8,191 tokens with 64 heads'
// queries 31.3 us, 0.72 of the copy's rate (FP8 cache: 31.6; a bare copy of pieces of 128
// bytes that lie apart takes 0.76 to 0.8 of it); 4 x 32,768 rows read back 49.2 us, 0.90
// (FP8, 0.78 of the bytes: 41 us, 0.84).  Few rows are bound by launch and by latencies one
// after another: the slot and position, the rows, the write (one token 3.7 us; 255 tokens 7,
// or 3.7 where L2 holds their rows already), or the starts, the search among them (a load
// a step), the table, the rows (five sequences 6 to 7).
#include "pa_codec.cuh"
#include "pa_latent.cuh"
#include "pa_rotate.cuh"

namespace pa {
namespace lat {
namespace {

using namespace codec;
using namespace rotary;

constexpr int kCtas = 28;   // one-warp CTAs per SM

struct AppendGrid {
  int parts, steps_per_part;
};

// fp32 -> the cache's bf16 value: over the scale where there is one
__device__ __forceinline__ void over_scale(float (&x)[8], float g) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = g > 0.f ? __fdiv_rn(x[i], g) : 0.f;
}

template <bool FP8, bool IL>
__global__ void __launch_bounds__(32, kCtas) append_kernel(const LatentAppendParams p, const AppendGrid gr) {
  const int lane = threadIdx.x, sub = lane >> 2, j = lane & 3;
  const int t = blockIdx.x / gr.parts, part = blockIdx.x % gr.parts;
  const int rows = p.Hq + 1;                          // every head's query, and the key's part
  const int s0 = part * gr.steps_per_part, s1 = min(1 + (rows + 7) / 8, s0 + gr.steps_per_part);
  struct Step {
    int h;                                            // -1: the latent
    uint4 a, b;
  };
  auto load = [&](int s) {
    Step x;
    x.h = s == 0 ? -1 : (s - 1) * 8 + sub;
    x.a = x.b = make_uint4(0, 0, 0, 0);
    if (s < s1) {
      if (s == 0) {
        const uint4 *src = reinterpret_cast<const uint4 *>(p.latent + (size_t)t * p.latent_stride);
        x.a = __ldg(src + lane);
        x.b = __ldg(src + 32 + lane);
      } else if (x.h < rows) {
        const uint4 *src = reinterpret_cast<const uint4 *>(
            x.h < p.Hq ? p.q + (size_t)t * p.q_stride + (size_t)x.h * p.q_head : p.rope + (size_t)t * p.rope_stride);
        x.a = src[j];     // (q_out may be q: not through the read-only path)
        x.b = src[j + 4];
      }
    }
    return x;
  };
  Step x0 = load(s0);
  float cs[8], sn[8];
  const int pos = __ldg(p.positions + t);
  const int64_t slot = __ldg(p.slots + t);
  if (s1 > 1) {
    float c, n;                                       // of pair `lane`
    angle(__ldg(p.inv_freq + lane), pos, p.factor, c, n);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int pair = IL ? (i < 4 ? 4 * j + i : 12 + 4 * j + i) : 8 * j + i;
      cs[i] = __shfl_sync(0xffffffffu, c, pair);
      sn[i] = __shfl_sync(0xffffffffu, n, pair);
    }
  }
  const bool bad = slot < -1 || slot >= (int64_t)p.kv.num_blocks * kBlock;
  if (bad && part == 0 && lane == 0) set_err(p.hdr, PA_ERRF_BAD_SLOT);
  const bool keep = slot >= 0 && !bad;
#pragma unroll 1
  for (int s = s0; s < s1; ++s) {
    const Step y = x0;
    x0 = load(s + 1);
    Pair16 x;
    unpack8(y.a, x.a);
    unpack8(y.b, x.b);
    if (y.h < 0) {
      if (p.norm) {
        const uint4 *w = reinterpret_cast<const uint4 *>(p.norm);
        rms_norm<512>(x, __ldg(w + lane), __ldg(w + 32 + lane), p.eps);
      }
      if (keep) {
        if constexpr (FP8) {
          uint2 *dst = reinterpret_cast<uint2 *>(static_cast<uint8_t *>(const_cast<void *>(p.kv.latent)) + slot * kLatent);
          dst[lane] = fp8_codes8(x.a, p.kv.g);
          dst[32 + lane] = fp8_codes8(x.b, p.kv.g);
        } else {
          uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(const_cast<void *>(p.kv.latent)) + slot * kLatent);
          dst[lane] = pack8(x.a);
          dst[32 + lane] = pack8(x.b);
        }
      }
      continue;
    }
    rotate<IL>(x, cs, sn, true, true);
    uint4 *dst = nullptr;
    if (y.h < p.Hq) {
      dst = reinterpret_cast<uint4 *>(p.q_out + (size_t)t * p.qo_stride + (size_t)y.h * p.qo_head);
    } else if (y.h == p.Hq && keep) {
      dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(const_cast<void *>(p.kv.rope)) + slot * kRope);
      if constexpr (FP8) {
        over_scale(x.a, p.kv.g);
        over_scale(x.b, p.kv.g);
      }
    }
    if (dst) {
      dst[j] = pack8(x.a);
      dst[j + 4] = pack8(x.b);
    }
  }
}

// ---------------------------------------------------------------- read-back

constexpr int kRowsPerWarp = 4;

template <bool FP8>
__global__ void __launch_bounds__(128) gather_kernel(const LatentGatherParams p) {
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && p.hdr)
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
      const int a = __ldg(p.starts + b), e = __ldg(p.starts + b + 1);
      if (a < 0 || e < a || e > p.N) set_err(p.hdr, PA_ERRF_BAD_Q_START);
    }
  const int row0 = (blockIdx.x * 4 + (threadIdx.x >> 5)) * kRowsPerWarp;
  if (row0 >= p.N) return;
  // lanes 0-3: the row's sequence (the last start at or before it), token and page
  int at = -2;   // slot in the pool; -1: zeros, -2: the row is left alone
  const int row = row0 + lane;
  if (lane < kRowsPerWarp && row < p.N && row >= __ldg(p.starts) && row < __ldg(p.starts + p.B)) {
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.starts + mid) <= row) lo = mid;
      else hi = mid;
    }
    const long long token = (long long)row - __ldg(p.starts + lo) + (p.first ? __ldg(p.first + lo) : 0);
    at = -1;
    if (token < 0) {
      set_err(p.hdr, PA_ERRF_NEG_LEN);
    } else if (token >= (long long)p.stride * kBlock) {
      set_err(p.hdr, PA_ERRF_LEN_OVER_CAPACITY);
    } else {
      const int id = __ldg(p.tables + (size_t)lo * p.stride + token / kBlock);
      if (id < 0 || id >= p.kv.num_blocks) set_err(p.hdr, PA_ERRF_BAD_BLOCK_ID);
      else at = id * kBlock + (int)(token % kBlock);
    }
  }
  constexpr int NC = FP8 ? 1 : 2;   // 16-byte pieces a lane of a row
  uint4 c[kRowsPerWarp][NC];
  uint4 r = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    const int a = __shfl_sync(0xffffffffu, at, i);
    const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.kv.latent) +
                                                       (size_t)max(a, 0) * (FP8 ? kLatent : 2 * kLatent));
#pragma unroll
    for (int k = 0; k < NC; ++k) c[i][k] = a >= 0 ? __ldg(src + k * 32 + lane) : make_uint4(0, 0, 0, 0);
  }
  const int ra = __shfl_sync(0xffffffffu, at, lane >> 3);   // eight lanes a row's rotated part
  if (ra >= 0) r = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.kv.rope) + (size_t)ra * kRope) + (lane & 7));
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    if (__shfl_sync(0xffffffffu, at, i) == -2) continue;
    uint4 *dst = reinterpret_cast<uint4 *>(p.latent_out + (size_t)(row0 + i) * kLatent);
    if constexpr (FP8) {
      const uint32_t w[4] = {c[i][0].x, c[i][0].y, c[i][0].z, c[i][0].w};
      float x[16];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 a = h2u_to_f2(e4m3x2_u16_to_h2(w[k] & 0xFFFFu)), b = h2u_to_f2(e4m3x2_u16_to_h2(w[k] >> 16));
        x[4 * k] = a.x * p.kv.g;
        x[4 * k + 1] = a.y * p.kv.g;
        x[4 * k + 2] = b.x * p.kv.g;
        x[4 * k + 3] = b.y * p.kv.g;
      }
      dst[2 * lane] = make_uint4(pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]), pack_bf2(x[4], x[5]), pack_bf2(x[6], x[7]));
      dst[2 * lane + 1] = make_uint4(pack_bf2(x[8], x[9]), pack_bf2(x[10], x[11]), pack_bf2(x[12], x[13]), pack_bf2(x[14], x[15]));
    } else {
#pragma unroll
      for (int k = 0; k < NC; ++k) dst[k * 32 + lane] = c[i][k];
    }
  }
  if (ra != -2) {
    if constexpr (FP8) {
      float x[8];
      unpack8(r, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= p.kv.g;
      r = pack8(x);
    }
    reinterpret_cast<uint4 *>(p.rope_out + (size_t)(row0 + (lane >> 3)) * kRope)[lane & 7] = r;
  }
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendParams &p, cudaStream_t s) {
  const int steps = 1 + (p.Hq + 1 + 7) / 8;
  // few tokens: a token's steps are spread over several warps, about sixteen warps an SM
  const int want = (2432 + p.T - 1) / p.T;
  AppendGrid gr;
  gr.parts = want < 1 ? 1 : want > steps ? steps : want;
  gr.steps_per_part = (steps + gr.parts - 1) / gr.parts;
  gr.parts = (steps + gr.steps_per_part - 1) / gr.steps_per_part;
  const unsigned grid = (unsigned)p.T * (unsigned)gr.parts;   // below 2^30 (rows are)
  const bool fp8 = p.kv.dtype == PA_KV_FP8;
  if (fp8 && p.interleaved) append_kernel<true, true><<<grid, 32, 0, s>>>(p, gr);
  else if (fp8) append_kernel<true, false><<<grid, 32, 0, s>>>(p, gr);
  else if (p.interleaved) append_kernel<false, true><<<grid, 32, 0, s>>>(p, gr);
  else append_kernel<false, false><<<grid, 32, 0, s>>>(p, gr);
  return cudaGetLastError();
}

cudaError_t launch_latent_gather(const LatentGatherParams &p, cudaStream_t s) {
  const unsigned grid = (unsigned)((p.N + 4LL * kRowsPerWarp - 1) / (4 * kRowsPerWarp));
  if (p.kv.dtype == PA_KV_FP8) gather_kernel<true><<<grid, 128, 0, s>>>(p);
  else gather_kernel<false><<<grid, 128, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace lat
}  // namespace pa
