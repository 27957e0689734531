// pa_latent_decode.cu -- the absorbed form of latent attention over the paged
// cache, the simplest kernel: a warp per (token, head), one key after another
// with the running maximum and sum of the softmax.
#include "pa_latent.cuh"

namespace pa {
namespace lat {
namespace {

template <bool FP8>
__global__ void __launch_bounds__(256) decode_kernel(const AbsorbedParams p) {
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= (long long)p.B * p.Q * p.H) return;
  const int bi = (int)(row / p.H), b = bi / p.Q, i = bi % p.Q;
  const int capacity = (int)min((long long)p.stride * kBlock, 0x7fffffffLL);
  int n = __ldg(p.seq_lens + b);
  if (row % ((long long)p.Q * p.H) == 0 && lane == 0 && n != 0 && (n < p.Q || n > capacity))
    set_err(p.hdr, n < 0 ? PA_ERRF_NEG_LEN : n < p.Q ? PA_ERRF_LEN_LT_QLEN : PA_ERRF_LEN_OVER_CAPACITY);
  n = min(max(n, 0), capacity);
  const int see = max(n - p.Q + 1 + i, 0);
  const __nv_bfloat16 *q = p.q + (size_t)row * kRow;
  float qv[18], o[16] = {}, top = kNegInf, sum = 0.f;
#pragma unroll
  for (int d = 0; d < 18; ++d) qv[d] = __bfloat162float(q[d * 32 + lane]);
  for (int t = 0; t < see; ++t) {
    const int id = __ldg(p.tables + (size_t)b * p.stride + t / kBlock);
    if (id < 0 || id >= p.kv.num_blocks) {
      if (lane == 0) set_err(p.hdr, PA_ERRF_BAD_BLOCK_ID);
      continue;
    }
    const size_t slot = (size_t)id * kBlock + t % kBlock;
    float c[18], s = 0.f;
#pragma unroll
    for (int d = 0; d < 16; ++d) {
      if constexpr (FP8)
        c[d] = h2u_to_f2(e4m3x2_u16_to_h2(static_cast<const uint8_t *>(p.kv.latent)[slot * kLatent + d * 32 + lane])).x;
      else
        c[d] = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.kv.latent)[slot * kLatent + d * 32 + lane]);
    }
#pragma unroll
    for (int d = 0; d < 2; ++d)
      c[16 + d] = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.kv.rope)[slot * kRope + d * 32 + lane]);
#pragma unroll
    for (int d = 0; d < 18; ++d) s += qv[d] * c[d];
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale_log2 * p.kv.g;
    const float mn = fmaxf(top, s), al = mn == kNegInf ? 1.f : exp2f(top - mn);
    const float w = exp2f(s - (mn == kNegInf ? 0.f : mn));
    top = mn;
    sum = sum * al + w;
#pragma unroll
    for (int d = 0; d < 16; ++d) o[d] = o[d] * al + w * c[d];
  }
  const float inv = sum != 0.f ? p.kv.g / sum : 0.f;
#pragma unroll
  for (int d = 0; d < 16; ++d) {
    const size_t at = (size_t)row * kLatent + d * 32 + lane;
    if (p.out_fp32) static_cast<float *>(p.out)[at] = o[d] * inv;
    else static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(o[d] * inv);
  }
  if (p.lse_out && lane == 0) p.lse_out[row] = sum != 0.f ? (top + log2f(sum)) * 0.69314718055994531f : kNegInf;
}

}  // namespace

cudaError_t launch_latent_decode(const AbsorbedParams &p, cudaStream_t s) {
  const unsigned grid = (unsigned)(((long long)p.B * p.Q * p.H + 7) / 8);
  if (p.kv.dtype == PA_KV_FP8) decode_kernel<true><<<grid, 256, 0, s>>>(p);
  else decode_kernel<false><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace lat
}  // namespace pa
