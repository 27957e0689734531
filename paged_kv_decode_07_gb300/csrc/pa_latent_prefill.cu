// pa_latent_prefill.cu -- the expanded form of latent attention over a ragged
// batch, the simplest kernel: a warp per (token, head), one key after another
// with the running maximum and sum of the softmax.
#include "pa_latent.cuh"

namespace pa {
namespace lat {
namespace {

__global__ void __launch_bounds__(256) prefill_kernel(const ExpandedParams p) {
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= (long long)p.T * p.H) return;
  const int t = (int)(row / p.H), h = (int)(row % p.H);
  auto qs = [&](int b) { return min(max(__ldg(p.q_starts + b), 0), p.T); };
  if (row == 0)
    for (int b = lane; b < p.B; b += 32) {
      const int a = __ldg(p.q_starts + b), e = __ldg(p.q_starts + b + 1);
      const int c = __ldg(p.kv_starts + b), d = __ldg(p.kv_starts + b + 1);
      if (a < 0 || e < a || e > p.T || c < 0 || d < c || d > p.N) set_err(p.hdr, PA_ERRF_BAD_Q_START);
      else if (p.causal && d > c && e - a > d - c) set_err(p.hdr, PA_ERRF_LEN_LT_QLEN);
    }
  if (t < qs(0) || t >= qs(p.B)) return;
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (qs(mid) <= t) lo = mid;
    else hi = mid;
  }
  const int k0 = min(max(__ldg(p.kv_starts + lo), 0), p.N), k1 = min(max(__ldg(p.kv_starts + lo + 1), k0), p.N);
  const int n = k1 - k0, m = qs(lo + 1) - qs(lo), i = t - qs(lo);
  const int see = p.causal ? min(max(n - m + 1 + i, 0), n) : n;
  const __nv_bfloat16 *q = p.q + (size_t)t * p.q_stride + (size_t)h * p.q_head;
  float qv[6], o[4] = {}, top = kNegInf, sum = 0.f;
#pragma unroll
  for (int d = 0; d < 6; ++d) qv[d] = __bfloat162float(q[d * 32 + lane]);
  for (int k = 0; k < see; ++k) {
    const __nv_bfloat16 *kn = p.kn + (size_t)(k0 + k) * p.k_stride + (size_t)h * p.k_head;
    const __nv_bfloat16 *kr = p.kr + (size_t)(k0 + k) * p.kr_stride;
    const __nv_bfloat16 *v = p.v + (size_t)(k0 + k) * p.v_stride + (size_t)h * p.v_head;
    float s = 0.f;
#pragma unroll
    for (int d = 0; d < 4; ++d) s += qv[d] * __bfloat162float(kn[d * 32 + lane]);
#pragma unroll
    for (int d = 0; d < 2; ++d) s += qv[4 + d] * __bfloat162float(kr[d * 32 + lane]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.scale_log2;
    const float mn = fmaxf(top, s), al = mn == kNegInf ? 1.f : exp2f(top - mn);
    const float w = exp2f(s - (mn == kNegInf ? 0.f : mn));
    top = mn;
    sum = sum * al + w;
#pragma unroll
    for (int d = 0; d < 4; ++d) o[d] = o[d] * al + w * __bfloat162float(v[d * 32 + lane]);
  }
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const size_t at = (size_t)row * kV + d * 32 + lane;
    if (p.out_fp32) static_cast<float *>(p.out)[at] = o[d] * inv;
    else static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(o[d] * inv);
  }
  if (p.lse_out && lane == 0) p.lse_out[row] = sum != 0.f ? (top + log2f(sum)) * 0.69314718055994531f : kNegInf;
}

}  // namespace

cudaError_t launch_latent_prefill(const ExpandedParams &p, cudaStream_t s) {
  prefill_kernel<<<(unsigned)(((long long)p.T * p.H + 7) / 8), 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace lat
}  // namespace pa
