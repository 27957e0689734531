// pa_prefill.cu -- ragged prefill: the choice of key splits, the attention
// kernel of the cache's format, and the join of what was split.
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

namespace {
// CTAs at once: one per SM of this GPU.  (Another count would only split the work
// worse: pieces, their workspace and their join go by this number alone.)
constexpr int kSms = 152;
int rows_of(int D) { return D == 128 ? 256 : 128; }
long long most_tiles(int T, int B, int Hkv, int G, int D) {
  return ((long long)T * G / rows_of(D) + B) * Hkv;
}
}  // namespace

// Key splits per row tile: one unless the row tiles leave half of the SMs
// idle; a split has at least 256 keys.
int prefill_splits(int T, int B, int Hkv, int G, int D, int max_seq_len) {
  const long long ctas = most_tiles(T, B, Hkv, G, D);
  const long long most = (max_seq_len + 255) / 256;
  long long s = kSms / (ctas > 0 ? ctas : 1);
  s = s < most ? s : most;
  return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}

// Where there may be more row tiles than SMs, the tiles of a last round that
// fills at most half of them are split over the others (768 tiles of 224 to
// 256 key tiles, six rounds of which the last had eight tiles: 2.33 -> 1.99
// ms; half as long, FP8: 619 -> 579 us).  Not where the tiles differ much
// (chunks of over half the keys they see: the longest first already even out),
// are short (below 64 key tiles the pieces and their join cost what they save;
// four packed prompts of 2 to 16 tiles: 58 -> 67 us),
// or come from more than 32 sequences (whose tiles are not counted).
int prefill_tail(int T, int B, int Hkv, int G, int D, int max_seq_len, int window) {
  long long span = max_seq_len;   // keys a row sees at most
  if (window > 0 && window < span) span = window;
  if (span < 64 * 128 || 2LL * T > span * B || B > 32) return 0;
  return most_tiles(T, B, Hkv, G, D) > kSms ? kSms : 0;
}
// partial rows of such a round
long long prefill_tail_rows(int D) { return (long long)kSms * rows_of(D); }

cudaError_t launch_prefill(const PrefillParams &p, cudaStream_t s) {
  const bool d128 = p.kv.D == 128;
  cudaError_t e = cudaErrorInvalidValue;
  switch (p.kv.dtype) {
    case PA_KV_BF16: e = d128 ? launch_prefill_bf16_d128(p, s) : launch_prefill_bf16_d256(p, s); break;
    case PA_KV_INT8: e = d128 ? launch_prefill_int8_d128(p, s) : launch_prefill_int8_d256(p, s); break;
    case PA_KV_NVFP4: e = d128 ? launch_prefill_nvfp4_d128(p, s) : launch_prefill_nvfp4_d256(p, s); break;
    case PA_KV_FP8: e = d128 ? launch_prefill_fp8_d128(p, s) : launch_prefill_fp8_d256(p, s); break;
  }
  if (e != cudaSuccess) return e;
  if (p.splits > 1) {
    const unsigned grid = (unsigned)(((long long)p.T * p.Hq + 7) / 8);
    return d128 ? launch_pdl(pf::prefill_join_kernel<128>, grid, 256, 0, s, p)
                : launch_pdl(pf::prefill_join_kernel<256>, grid, 256, 0, s, p);
  }
  if (p.tail > 0)
    return d128 ? launch_pdl(pf::prefill_join_tail_kernel<128>, kSms, 256, 0, s, p)
                : launch_pdl(pf::prefill_join_tail_kernel<256>, kSms, 256, 0, s, p);
  return cudaSuccess;
}

}  // namespace pa
