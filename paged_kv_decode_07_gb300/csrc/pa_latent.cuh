// pa_latent.cuh -- what the kernels of latent attention share with their host
// side (pa_latent_api.cu): parameters, sizes, launches.
#pragma once

#include "pa_internal.cuh"

namespace pa {
namespace lat {

constexpr int kLatent = 512;          // latent values of a token
constexpr int kRope = 64;             // rotated values
constexpr int kRow = kLatent + kRope; // of an absorbed query
constexpr int kNope = 128;            // expanded: key dims of a head beside the rotated ones,
constexpr int kQk = kNope + kRope;    // all of them,
constexpr int kV = 128;               // and value dims
constexpr int kMaxHeads = 128;
// CTAs at once: one per SM of this GPU (another count would only split the work worse)
constexpr int kSms = 152;

struct LatentView {
  int dtype, num_blocks;
  const void *latent, *rope;
  float g;                            // value = stored * g (bf16: 1)
};

struct LatentAppendParams {
  LatentView kv;
  int T, Hq;
  const __nv_bfloat16 *latent, *rope, *q;
  __nv_bfloat16 *q_out;
  long long latent_stride, rope_stride, q_stride, q_head, qo_stride, qo_head;
  const int *positions;
  const int64_t *slots;
  int interleaved;
  const float *inv_freq;
  float factor, eps;
  const __nv_bfloat16 *norm;
  uint32_t *hdr;
};

struct LatentGatherParams {
  LatentView kv;
  const int *tables;
  int stride;
  const int *starts, *first;
  int B, N;
  __nv_bfloat16 *latent_out, *rope_out;
  uint32_t *hdr;
};

struct ExpandedParams {
  int B, H, T, N;                     // sequences, heads, query rows, key rows
  const __nv_bfloat16 *q, *kn, *kr, *v;
  long long q_stride, q_head, k_stride, k_head, kr_stride, v_stride, v_head;
  const int *q_starts, *kv_starts;
  int causal;
  float scale_log2;                   // softmax_scale * log2(e)
  void *out;
  int out_fp32;
  float *lse_out;
  uint32_t *hdr;
  int shares;                         // places of the kernel's list of work
  // partial outputs of items in pieces: [item][piece][256][128] and their lse, or null
  float *part_o;
  float *part_lse;
};

struct AbsorbedParams {
  LatentView kv;
  const __nv_bfloat16 *q;             // [B, Q, H, 576]
  int B, Q, H;
  const int *tables;
  int stride;
  const int *seq_lens;
  float scale_log2;
  void *out;
  int out_fp32;
  float *lse_out;
  uint32_t *hdr;
  // work: see DecodePlan
  int R, RG, S, workers, least;       // least: tiles of a run
  uint32_t *flags;                    // [workers * S]
  int *starts;                        // [B + 1] tiles of the sequences before
  float *part_o;                      // [2 * workers][S][R][512]
  float *part_lse;                    // [2 * workers][S][R]
};

// The rows (token, head) of a sequence in RG groups of R, one CTA each; S groups
// walk the same keys side by side (a worker), RG / S such sets one after another.
// The key tiles of all sets of all sequences are one list, of which every worker
// takes an equal run.
constexpr int kMaxRows = 64;
struct DecodePlan {
  int R, RG, S, workers, least;
};
DecodePlan plan_latent_decode(int B, int Q, int H, int max_seq_len);

cudaError_t launch_latent_append(const LatentAppendParams &p, cudaStream_t s);
cudaError_t launch_latent_gather(const LatentGatherParams &p, cudaStream_t s);
long long latent_prefill_parts(int B, int H, int T, int N);
cudaError_t launch_latent_prefill(const ExpandedParams &p, cudaStream_t s);
cudaError_t launch_latent_decode(const AbsorbedParams &p, cudaStream_t s);

}  // namespace lat
}  // namespace pa
