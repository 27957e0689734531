// pa_prefill.cu -- ragged prefill: the choice of key splits, the attention
// kernel of the cache's format, and the join of the splits.
#include "pa_prefill.cuh"

namespace pa {

cudaError_t launch_prefill_bf16_d128(const PrefillParams &p, cudaStream_t s);
cudaError_t launch_prefill_bf16_d256(const PrefillParams &p, cudaStream_t s);
cudaError_t launch_prefill_int8_d128(const PrefillParams &p, cudaStream_t s);
cudaError_t launch_prefill_int8_d256(const PrefillParams &p, cudaStream_t s);
cudaError_t launch_prefill_nvfp4_d128(const PrefillParams &p, cudaStream_t s);
cudaError_t launch_prefill_nvfp4_d256(const PrefillParams &p, cudaStream_t s);
cudaError_t launch_prefill_fp8_d128(const PrefillParams &p, cudaStream_t s);
cudaError_t launch_prefill_fp8_d256(const PrefillParams &p, cudaStream_t s);

// Key splits per row tile: one unless the row tiles leave half of the SMs
// idle; a split has at least 256 keys.
int prefill_splits(int T, int B, int Hkv, int G, int D, int max_seq_len) {
  const int rows = D == 128 ? 256 : 128;
  const long long ctas = ((long long)T * G / rows + B) * Hkv;
  const long long most = (max_seq_len + 255) / 256;
  long long s = 152 / (ctas > 0 ? ctas : 1);
  s = s < most ? s : most;
  return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}

cudaError_t launch_prefill(const PrefillParams &p, cudaStream_t s) {
  const bool d128 = p.kv.D == 128;
  cudaError_t e = cudaErrorInvalidValue;
  switch (p.kv.dtype) {
    case PA_KV_BF16: e = d128 ? launch_prefill_bf16_d128(p, s) : launch_prefill_bf16_d256(p, s); break;
    case PA_KV_INT8: e = d128 ? launch_prefill_int8_d128(p, s) : launch_prefill_int8_d256(p, s); break;
    case PA_KV_NVFP4: e = d128 ? launch_prefill_nvfp4_d128(p, s) : launch_prefill_nvfp4_d256(p, s); break;
    case PA_KV_FP8: e = d128 ? launch_prefill_fp8_d128(p, s) : launch_prefill_fp8_d256(p, s); break;
  }
  if (e != cudaSuccess || p.splits == 1) return e;
  const long long rows = (long long)p.T * p.Hq;
  const unsigned grid = (unsigned)((rows + 7) / 8);
  return d128 ? launch_pdl(pf::prefill_join_kernel<128>, grid, 256, 0, s, p)
              : launch_pdl(pf::prefill_join_kernel<256>, grid, 256, 0, s, p);
}

}  // namespace pa
