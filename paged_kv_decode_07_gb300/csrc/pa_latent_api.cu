// pa_latent_api.cu -- host side of the latent-attention entry points of
// include/pa.h: argument checks (nothing is launched when one fails),
// workspace layout and launches.
#include <cmath>
#include <cstring>

#include "pa_latent.cuh"
#include "pa_launch.h"

using namespace pa;
using namespace pa::lat;

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned8(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int check_cache(const pa_latent_cache *kv) {
  if (!kv) return PA_ERR_INVALID_ARG;
  if (kv->dtype < PA_KV_BF16 || kv->dtype > PA_KV_FP8) return PA_ERR_INVALID_ARG;
  if (kv->dtype != PA_KV_BF16 && kv->dtype != PA_KV_FP8) return PA_ERR_UNSUPPORTED;
  if (kv->num_blocks < 1) return PA_ERR_INVALID_ARG;
  if (kv->block_size != kBlock || kv->latent_dim != kLatent || kv->rope_dim != kRope)
    return PA_ERR_UNSUPPORTED;
  if (kv->num_blocks > (1 << 27)) return PA_ERR_UNSUPPORTED;   // (slots and rows of the pool: 31 bits)
  if (!kv->latent || !kv->rope || !aligned16(kv->latent) || !aligned16(kv->rope)) return PA_ERR_INVALID_ARG;
  if (kv->dtype == PA_KV_FP8 && !std::isfinite(kv->global_scale)) return PA_ERR_INVALID_ARG;
  return PA_OK;
}

LatentView view_of(const pa_latent_cache *kv) {
  return {kv->dtype, kv->num_blocks, kv->latent, kv->rope, kv->dtype == PA_KV_FP8 ? kv->global_scale : 1.0f};
}

// a stride that a second token (or head) would need
bool stride_ok(int count, long long stride, long long least) {
  return count < 2 || (stride >= least && stride % 8 == 0);
}

// a call without work clears the flags of a workspace of its own (a pointer that
// is none is left alone: such a call reads no argument)
int nothing_to_do(void *ws, size_t ws_bytes, cudaStream_t s) {
  cudaPointerAttributes at;
  if (!ws || !aligned16(ws) || ws_bytes < kHdrWords * 4) return PA_OK;
  if (cudaPointerGetAttributes(&at, ws) != cudaSuccess) {
    (void)cudaGetLastError();
    return PA_OK;
  }
  if (at.type == cudaMemoryTypeUnregistered) return PA_OK;
  return cudaMemsetAsync(ws, 0, 16, s) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int check_prefill(const pa_latent_prefill_problem *p) {
  if (!p || p->batch < 0 || p->num_tokens < 0 || p->num_keys < 0 || p->num_heads < 1) return PA_ERR_INVALID_ARG;
  if (!std::isfinite(p->softmax_scale)) return PA_ERR_INVALID_ARG;
  // rows (token, head) and tiles stay within 32-bit indices
  if (((long long)p->num_tokens + p->batch) * p->num_heads > (1LL << 30) || p->batch > (1 << 24) ||
      p->num_keys > (1 << 30))
    return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

int check_decode(const pa_latent_problem *p) {
  if (!p || p->batch < 0 || p->max_seq_len < 0) return PA_ERR_INVALID_ARG;
  if (p->num_heads < 1 || p->q_len < 1) return PA_ERR_INVALID_ARG;
  if (p->num_heads > kMaxHeads || p->q_len > kMaxQLen) return PA_ERR_UNSUPPORTED;
  if (!std::isfinite(p->softmax_scale)) return PA_ERR_INVALID_ARG;
  if (p->batch > 0 && (p->block_table_stride < 1 || p->block_table_stride > (1 << 26))) return PA_ERR_INVALID_ARG;
  if ((long long)p->batch * p->q_len * p->num_heads > (1LL << 27)) return PA_ERR_UNSUPPORTED;
  // the key tiles of a call are counted in 32 bits
  const DecodePlan d = plan_latent_decode(p->batch, p->q_len, p->num_heads, p->max_seq_len);
  if (p->batch > 0 && (p->block_table_stride + 1LL) / 2 * p->batch * (d.RG / d.S) >= (1LL << 31)) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

struct DecodeLayout {
  DecodePlan plan;
  size_t flags, starts, part_lse, part_o, total;
};

DecodeLayout decode_layout(const pa_latent_problem *p) {
  DecodeLayout L;
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  L.plan = plan_latent_decode(p->batch, p->q_len, p->num_heads, p->max_seq_len);
  const size_t rows = (size_t)2 * L.plan.workers * L.plan.S * L.plan.R;
  L.flags = kHdrWords * 4;
  L.starts = L.flags + up((size_t)L.plan.workers * L.plan.S * 4);
  L.part_lse = L.starts + up(((size_t)p->batch + 1) * 4);
  L.part_o = L.part_lse + up(rows * 4);
  L.total = L.part_o + rows * kLatent * 4;
  return L;
}

}  // namespace

extern "C" {

int pa_latent_append(const pa_latent_cache *kv, const pa_latent_new *in, void *ws, pa_stream_t stream) {
  const int st = check_cache(kv);
  if (st) return st;
  if (!in || in->num_tokens < 0 || in->num_q_heads < 0) return PA_ERR_INVALID_ARG;
  if (ws && !aligned16(ws)) return PA_ERR_INVALID_ARG;
  if (!std::isfinite(in->attn_factor) || !std::isfinite(in->eps) || in->eps < 0.f) return PA_ERR_INVALID_ARG;
  if ((long long)in->num_tokens * (in->num_q_heads + 8LL) > (1LL << 30)) return PA_ERR_UNSUPPORTED;
  const int T = in->num_tokens, Hq = in->num_q_heads;
  if (T > 0) {
    if (!in->latent || !in->rope || !in->positions || !in->slot_mapping || !in->inv_freq) return PA_ERR_INVALID_ARG;
    if (!aligned16(in->latent) || !aligned16(in->rope) || !aligned16(in->norm) || !aligned4(in->positions) ||
        !aligned4(in->inv_freq) || !aligned8(in->slot_mapping))
      return PA_ERR_INVALID_ARG;
    if (!stride_ok(T, in->latent_stride, 0) || !stride_ok(T, in->rope_stride, 0)) return PA_ERR_INVALID_ARG;
    if (Hq > 0) {
      if (!in->q || !in->q_out || !aligned16(in->q) || !aligned16(in->q_out)) return PA_ERR_INVALID_ARG;
      if (!stride_ok(T, in->q_stride, 0) || !stride_ok(Hq, in->q_head_stride, 0) ||
          !stride_ok(T, in->q_out_stride, kRope) || !stride_ok(Hq, in->q_out_head_stride, kRope))
        return PA_ERR_INVALID_ARG;
    }
  }
  uint32_t *hdr = static_cast<uint32_t *>(ws);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (hdr && cudaMemsetAsync(hdr, 0, 4, s) != cudaSuccess) return PA_ERR_CUDA;
  if (T == 0) return PA_OK;
  LatentAppendParams p;
  std::memset(&p, 0, sizeof p);
  p.kv = view_of(kv);
  p.T = T;
  p.Hq = Hq;
  p.latent = static_cast<const __nv_bfloat16 *>(in->latent);
  p.rope = static_cast<const __nv_bfloat16 *>(in->rope);
  p.q = static_cast<const __nv_bfloat16 *>(in->q);
  p.q_out = static_cast<__nv_bfloat16 *>(in->q_out);
  p.latent_stride = in->latent_stride;
  p.rope_stride = in->rope_stride;
  p.q_stride = in->q_stride;
  p.q_head = in->q_head_stride;
  p.qo_stride = in->q_out_stride;
  p.qo_head = in->q_out_head_stride;
  p.positions = in->positions;
  p.slots = in->slot_mapping;
  p.interleaved = in->interleaved ? 1 : 0;
  p.inv_freq = in->inv_freq;
  p.factor = in->attn_factor;
  p.eps = in->eps;
  p.norm = static_cast<const __nv_bfloat16 *>(in->norm);
  p.hdr = hdr;
  return launch_latent_append(p, s) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int pa_latent_gather(const pa_latent_cache *kv, const int32_t *block_tables, int32_t block_table_stride,
                     const int32_t *starts, const int32_t *first, int32_t batch, int32_t num_rows,
                     void *latent_out, void *rope_out, void *ws, pa_stream_t stream) {
  const int st = check_cache(kv);
  if (st) return st;
  if (batch < 0 || num_rows < 0 || (ws && !aligned16(ws))) return PA_ERR_INVALID_ARG;
  if (num_rows > (1 << 30) || batch > (1 << 24)) return PA_ERR_UNSUPPORTED;
  uint32_t *hdr = static_cast<uint32_t *>(ws);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (batch > 0 && num_rows > 0) {
    if (!block_tables || !starts || !latent_out || !rope_out) return PA_ERR_INVALID_ARG;
    if (block_table_stride < 1 || block_table_stride > (1 << 26)) return PA_ERR_INVALID_ARG;
    if (!aligned4(block_tables) || !aligned4(starts) || !aligned4(first) || !aligned16(latent_out) ||
        !aligned16(rope_out))
      return PA_ERR_INVALID_ARG;
  }
  if (hdr && cudaMemsetAsync(hdr, 0, 4, s) != cudaSuccess) return PA_ERR_CUDA;
  if (batch == 0 || num_rows == 0) return PA_OK;
  LatentGatherParams p;
  std::memset(&p, 0, sizeof p);
  p.kv = view_of(kv);
  p.tables = block_tables;
  p.stride = block_table_stride;
  p.starts = starts;
  p.first = first;
  p.B = batch;
  p.N = num_rows;
  p.latent_out = static_cast<__nv_bfloat16 *>(latent_out);
  p.rope_out = static_cast<__nv_bfloat16 *>(rope_out);
  p.hdr = hdr;
  return launch_latent_gather(p, s) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

size_t pa_latent_prefill_workspace_bytes(const pa_latent_prefill_problem *p) {
  if (check_prefill(p) != PA_OK) return 0;
  return kHdrWords * 4 + (size_t)latent_prefill_parts(p->batch, p->num_heads, p->num_tokens, p->num_keys) * (kV + 1) * 4;
}

int pa_latent_prefill(const pa_latent_prefill_problem *p, void *ws, size_t ws_bytes, pa_stream_t stream) {
  const int st = check_prefill(p);
  if (st) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (p->batch == 0 || p->num_tokens == 0) return nothing_to_do(ws, ws_bytes, s);
  if (!p->q || !p->q_starts || !p->kv_starts || !p->out) return PA_ERR_INVALID_ARG;
  if (p->num_keys > 0 && (!p->k_nope || !p->k_rope || !p->v)) return PA_ERR_INVALID_ARG;
  if (!aligned16(p->q) || !aligned16(p->k_nope) || !aligned16(p->k_rope) || !aligned16(p->v) ||
      !aligned16(p->out) || !aligned4(p->q_starts) || !aligned4(p->kv_starts) || !aligned4(p->lse_out))
    return PA_ERR_INVALID_ARG;
  if (!stride_ok(p->num_tokens, p->q_stride, 8) || !stride_ok(p->num_heads, p->q_head_stride, 8) ||
      !stride_ok(p->num_keys, p->k_stride, 8) || !stride_ok(p->num_heads, p->k_head_stride, 8) ||
      !stride_ok(p->num_keys, p->k_rope_stride, 8) || !stride_ok(p->num_keys, p->v_stride, 8) ||
      !stride_ok(p->num_heads, p->v_head_stride, 8))
    return PA_ERR_INVALID_ARG;
  if (!ws || !aligned16(ws)) return PA_ERR_INVALID_ARG;
  if (ws_bytes < pa_latent_prefill_workspace_bytes(p)) return PA_ERR_WORKSPACE_TOO_SMALL;
  ExpandedParams a;
  std::memset(&a, 0, sizeof a);
  a.B = p->batch;
  a.H = p->num_heads;
  a.T = p->num_tokens;
  a.N = p->num_keys;
  a.q = static_cast<const __nv_bfloat16 *>(p->q);
  a.kn = static_cast<const __nv_bfloat16 *>(p->k_nope);
  a.kr = static_cast<const __nv_bfloat16 *>(p->k_rope);
  a.v = static_cast<const __nv_bfloat16 *>(p->v);
  a.q_stride = p->q_stride;
  a.q_head = p->q_head_stride;
  a.k_stride = p->k_stride;
  a.k_head = p->k_head_stride;
  a.kr_stride = p->k_rope_stride;
  a.v_stride = p->v_stride;
  a.v_head = p->v_head_stride;
  a.q_starts = p->q_starts;
  a.kv_starts = p->kv_starts;
  a.causal = p->causal ? 1 : 0;
  a.scale_log2 = p->softmax_scale * 1.4426950408889634f;
  a.out = p->out;
  a.out_fp32 = p->out_fp32 ? 1 : 0;
  a.lse_out = p->lse_out;
  a.hdr = static_cast<uint32_t *>(ws);
  if (const long long rows = latent_prefill_parts(p->batch, p->num_heads, p->num_tokens, p->num_keys)) {
    a.part_o = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + kHdrWords * 4);
    a.part_lse = a.part_o + rows * kV;
  }
  if (launch_clear(a.hdr, s) != cudaSuccess) return PA_ERR_CUDA;
  return launch_latent_prefill(a, s) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

size_t pa_latent_decode_workspace_bytes(const pa_latent_cache *kv, const pa_latent_problem *p) {
  return check_cache(kv) == PA_OK && check_decode(p) == PA_OK ? decode_layout(p).total : 0;
}

int pa_latent_decode(const pa_latent_cache *kv, const pa_latent_problem *p, void *ws, size_t ws_bytes,
                     pa_stream_t stream) {
  int st = check_cache(kv);
  if (st) return st;
  st = check_decode(p);
  if (st) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (p->batch == 0) return nothing_to_do(ws, ws_bytes, s);
  if (!p->q || !p->block_tables || !p->seq_lens || !p->out) return PA_ERR_INVALID_ARG;
  if (!aligned16(p->q) || !aligned16(p->out) || !aligned4(p->block_tables) || !aligned4(p->seq_lens) ||
      !aligned4(p->lse_out))
    return PA_ERR_INVALID_ARG;
  if (!ws || !aligned16(ws)) return PA_ERR_INVALID_ARG;
  const DecodeLayout L = decode_layout(p);
  if (ws_bytes < L.total) return PA_ERR_WORKSPACE_TOO_SMALL;
  uint8_t *w = static_cast<uint8_t *>(ws);
  AbsorbedParams a;
  std::memset(&a, 0, sizeof a);
  a.kv = view_of(kv);
  a.q = static_cast<const __nv_bfloat16 *>(p->q);
  a.B = p->batch;
  a.Q = p->q_len;
  a.H = p->num_heads;
  a.tables = p->block_tables;
  a.stride = p->block_table_stride;
  a.seq_lens = p->seq_lens;
  a.scale_log2 = p->softmax_scale * 1.4426950408889634f;
  a.out = p->out;
  a.out_fp32 = p->out_fp32 ? 1 : 0;
  a.lse_out = p->lse_out;
  a.hdr = static_cast<uint32_t *>(ws);
  a.R = L.plan.R;
  a.RG = L.plan.RG;
  a.S = L.plan.S;
  a.workers = L.plan.workers;
  a.least = L.plan.least;
  a.flags = reinterpret_cast<uint32_t *>(w + L.flags);
  a.starts = reinterpret_cast<int *>(w + L.starts);
  a.part_lse = reinterpret_cast<float *>(w + L.part_lse);
  a.part_o = reinterpret_cast<float *>(w + L.part_o);
  return launch_latent_decode(a, s) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // extern "C"
