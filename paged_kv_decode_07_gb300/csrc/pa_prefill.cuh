// pa_prefill.cuh -- parts of the ragged prefill shared by its translation
// units: the map from a tile index to a sequence's rows, and the join of key
// splits.
//
// A row is one (query token, query head) of a kv head's group: row r of a
// sequence is token r / G, head r % G, so that the G heads that share a kv
// head share every key tile that is read.
#pragma once

#include "pa_launch.h"
#include "pa_score.cuh"

namespace pa {
namespace pf {

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// sets a flag once the header has been cleared (the kernel before this one)
__device__ __forceinline__ void flag(uint32_t *hdr, uint32_t bits) {
  griddep_wait();
  set_err(hdr, bits);
}

// the sequence and row tile of tile index `tile` (tiles of all sequences in
// order, `per` tokens each): every thread of a warp gets the answer
struct TileOf {
  // sequence (-1: none), tile in it, its query rows' start and count, its keys
  int b, first, start, len, n;
};
__device__ __forceinline__ TileOf find_tile(const PrefillParams &p, int tile, int rows_per_tile) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  uint32_t err = 0;
  TileOf r = {-1, 0, 0, 0, 0};
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    int start = 0, len = 0, keys = 0;
    if (b < p.B) {
      const int s0 = __ldg(p.q_starts + b), s1 = __ldg(p.q_starts + b + 1);
      keys = __ldg(p.seq_lens + b);
      start = min(max(s0, 0), p.T);
      const int end = min(max(s1, start), p.T);
      if (start != s0 || end != s1) err = 1;
      len = end - start;
    }
    const int n = (int)(((long long)len * p.G + rows_per_tile - 1) / rows_per_tile);
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, before + inc > tile);
    if (hit) {
      const int l = __ffs(hit) - 1;
      r.b = b0 + l;
      r.first = tile - (before + __shfl_sync(0xffffffffu, inc - n, l));
      r.start = __shfl_sync(0xffffffffu, start, l);
      r.len = __shfl_sync(0xffffffffu, len, l);
      r.n = __shfl_sync(0xffffffffu, keys, l);
      break;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (err) flag(p.hdr, PA_ERRF_BAD_Q_START);
  return r;
}

// joins the key splits of every row of the batch's sequences: one warp a row
template <int D>
__global__ void __launch_bounds__(256) prefill_join_kernel(const PrefillParams p) {
  griddep_wait();   // the splits are complete
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const long long rows = (long long)p.T * p.Hq;
  if (row >= rows) return;
  const int t = (int)(row / p.Hq);
  const int lo = min(max(__ldg(p.q_starts), 0), p.T), hi = min(max(__ldg(p.q_starts + p.B), 0), p.T);
  if (t < lo || t >= hi) return;   // rows of no sequence stay as they were
  float M = kNegInf;
  for (int s = 0; s < p.splits; ++s) M = fmaxf(M, p.part_lse[s * rows + row]);
  float sum = 0.f, acc[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) acc[i] = 0.f;
  if (M != kNegInf)
    for (int s = 0; s < p.splits; ++s) {
      const float ls = p.part_lse[s * rows + row];
      if (ls == kNegInf) continue;
      const float w = expf(ls - M);
      sum += w;
      const float4 *src = reinterpret_cast<const float4 *>(p.part_o + (s * rows + row) * D);
#pragma unroll
      for (int i = 0; i < D / 128; ++i) {
        const float4 x = __ldcs(src + i * 32 + lane);
        acc[4 * i] += w * x.x;
        acc[4 * i + 1] += w * x.y;
        acc[4 * i + 2] += w * x.z;
        acc[4 * i + 3] += w * x.w;
      }
    }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
  for (int i = 0; i < D / 128; ++i) {
    const size_t at = (size_t)row * D + (i * 32 + lane) * 4;
    const float x[4] = {acc[4 * i] * inv, acc[4 * i + 1] * inv, acc[4 * i + 2] * inv, acc[4 * i + 3] * inv};
    if (p.out_fp32)
      *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) = make_float4(x[0], x[1], x[2], x[3]);
    else
      *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + at) =
          make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
  }
  if (lane == 0 && p.lse_out) p.lse_out[row] = sum > 0.f ? M + logf(sum) : kNegInf;
}


}  // namespace pf
}  // namespace pa
