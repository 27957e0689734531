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

// One CTA's share of the batch: a row tile of a sequence and kv head, and which
// of how many pieces of its keys.  The tiles of all sequences are counted in
// order (rows_per_tile rows each) and taken from the last: the last tokens of a
// prompt see most.  Pieces: all tiles in p.splits (few tiles), or, where the
// tiles fill the GPU several times and then a little more, those of the last
// round (p.tail: SMs) in as many pieces as make it a full round of short ones.
struct Share {
  int b;                      // sequence, -1: nothing to do
  int first, start, len, n;   // tile in it, its query rows' start and count, its keys
  int kvh, piece, pieces;
  int tail;                   // place among the tiles of the last round, -1: not one
};
struct Round {
  int tail, pieces;           // tiles in pieces at the end, pieces of each
};
__device__ __forceinline__ Round last_round(int total, int sms) {
  Round r = {0, 1};
  const int rem = sms > 0 ? total % sms : 0;
  if (total > sms && rem > 0 && 2 * rem <= sms) {
    r.tail = rem;
    r.pieces = min(16, sms / rem);
  }
  return r;
}

// More than 32 sequences: sequence b's tiles are given the places from
// q_starts[b] * G / rows + b on, of which there are enough (and at most one too
// many), so that a search finds a place's sequence (in two loads for 1,024
// sequences, three for 32,768) without the counts of those before it.  CTA 0
// looks at all starts.
__device__ __forceinline__ Share search_share(const PrefillParams &p, int index, int rows_per_tile) {
  const int lane = threadIdx.x & 31, Hkv = p.kv.hkv;
  Share r = {-1, 0, 0, 0, 0, 0, 0, 1, -1};
  auto start = [&](int b) { return min(max(__ldg(p.q_starts + b), 0), p.T); };
  auto place = [&](int b) { return (int)((long long)start(b) * p.G / rows_per_tile) + b; };
  if (index == 0) {
    bool bad = false;
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
      const int s0 = __ldg(p.q_starts + b), s1 = __ldg(p.q_starts + b + 1);
      bad = bad || s0 < 0 || s1 < s0 || s1 > p.T;
    }
    if (bad) flag(p.hdr, PA_ERRF_BAD_Q_START);
  }
  const int total = place(p.B);   // at most rows / rows_per_tile + B
  const int t = index / p.splits, at = total - 1 - t / Hkv;
  r.piece = index % p.splits;
  r.pieces = p.splits;
  r.kvh = t % Hkv;
  if (at < 0) return r;
  int lo = 0, hi = p.B;   // the last sequence of [lo, hi) that starts at or before `at`
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, b = lo + lane * step;
    const uint32_t le = __ballot_sync(0xffffffffu, b < hi && place(b) <= at);
    lo += (31 - __clz((int)(le | 1u))) * step;
    hi = min(hi, lo + step);
  }
  const int first = at - place(lo), s0 = start(lo), len = max(start(lo + 1) - s0, 0);
  if (first < 0 || (long long)first * rows_per_tile >= (long long)len * p.G) return r;
  r.b = lo;
  r.first = first;
  r.start = s0;
  r.len = len;
  r.n = __ldg(p.seq_lens + lo);
  return r;
}

// every thread of a warp gets the answer; `index`: of the CTA, or, in the join,
// of a tail tile (join = true)
__device__ __forceinline__ Share find_share(const PrefillParams &p, int index, int rows_per_tile, bool join) {
  if (p.B > 32) return search_share(p, index, rows_per_tile);   // (there is no tail then)
  const int lane = threadIdx.x & 31, Hkv = p.kv.hkv;
  // this lane's sequence, and the tiles up to it (inclusive)
  int start = 0, len = 0, keys = 0;
  if (lane < p.B) {
    const int s0 = __ldg(p.q_starts + lane), s1 = __ldg(p.q_starts + lane + 1);
    keys = __ldg(p.seq_lens + lane);
    start = min(max(s0, 0), p.T);
    const int end = min(max(s1, start), p.T);
    if ((start != s0 || end != s1) && !join) flag(p.hdr, PA_ERRF_BAD_Q_START);
    len = end - start;
  }
  const int n = (int)(((long long)len * p.G + rows_per_tile - 1) / rows_per_tile);
  int inc = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  Share r = {-1, 0, 0, 0, 0, 0, 0, 1, -1};
  // at most rows / rows_per_tile + B: the host bounds them by 2^30 (descending
  // starts count rows more than once, each sequence at most T)
  const int tiles = __shfl_sync(0xffffffffu, inc, 31);
  const int total = tiles * Hkv;
  const Round last = last_round(total, p.tail);
  int t = index;   // tile and kv head
  if (join) {
    if (index >= last.tail) return r;
    t = total - last.tail + index;
    r.tail = index;
    r.pieces = last.pieces;
  } else if (p.splits > 1) {
    r.piece = index % p.splits;
    r.pieces = p.splits;
    t = index / p.splits;
  } else if (last.tail > 0 && index >= total - last.tail) {
    const int x = index - (total - last.tail);
    r.tail = x / last.pieces;
    r.piece = x % last.pieces;
    r.pieces = last.pieces;
    t = total - last.tail + r.tail;
  }
  if (t >= total) return r;
  r.kvh = t % Hkv;
  const int tile = tiles - 1 - t / Hkv;
  const int l = __ffs(__ballot_sync(0xffffffffu, inc > tile)) - 1;
  r.b = l;
  r.first = tile - __shfl_sync(0xffffffffu, inc - n, l);
  r.start = __shfl_sync(0xffffffffu, start, l);
  r.len = __shfl_sync(0xffffffffu, len, l);
  r.n = __shfl_sync(0xffffffffu, keys, l);
  return r;
}

// out = sum_s w_s o_s / sum_s w_s of one row over `parts` partial rows
// `pitch` rows apart, w_s = exp(lse_s - max); one warp a row
template <int D>
__device__ __forceinline__ void join_row(const PrefillParams &p, size_t part, size_t pitch, int parts,
                                         size_t row, int lane) {
  float M = kNegInf;
  for (int s = 0; s < parts; ++s) M = fmaxf(M, p.part_lse[part + s * pitch]);
  float sum = 0.f, acc[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) acc[i] = 0.f;
  for (int s = 0; s < parts; ++s) {
    const float ls = p.part_lse[part + s * pitch];
    if (ls == kNegInf) continue;
    const float w = expf(ls - M);   // (a NaN among a part's scores is in its lse)
    sum += w;
    const float4 *src = reinterpret_cast<const float4 *>(p.part_o + (part + s * pitch) * D);
#pragma unroll
    for (int i = 0; i < D / 128; ++i) {
      const float4 x = __ldcs(src + i * 32 + lane);
      acc[4 * i] += w * x.x;
      acc[4 * i + 1] += w * x.y;
      acc[4 * i + 2] += w * x.z;
      acc[4 * i + 3] += w * x.w;
    }
  }
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll
  for (int i = 0; i < D / 128; ++i) {
    const size_t at = row * D + (i * 32 + lane) * 4;
    const float x[4] = {acc[4 * i] * inv, acc[4 * i + 1] * inv, acc[4 * i + 2] * inv, acc[4 * i + 3] * inv};
    if (p.out_fp32)
      *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) = make_float4(x[0], x[1], x[2], x[3]);
    else
      *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + at) =
          make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
  }
  if (lane == 0 && p.lse_out) p.lse_out[row] = sum != 0.f ? M + logf(sum) : kNegInf;
}

// all rows in p.splits pieces
template <int D>
__global__ void __launch_bounds__(256) prefill_join_kernel(const PrefillParams p) {
  griddep_wait();   // the pieces are complete
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const long long rows = (long long)p.T * p.Hq;
  if (row >= rows) return;
  const int t = (int)(row / p.Hq);
  const int lo = min(max(__ldg(p.q_starts), 0), p.T), hi = min(max(__ldg(p.q_starts + p.B), 0), p.T);
  if (t < lo || t >= hi) return;   // rows of no sequence stay as they were
  join_row<D>(p, (size_t)row, (size_t)rows, p.splits, (size_t)row, threadIdx.x & 31);
}

// the tiles of the last round, eight rows at a time over all CTAs
template <int D>
__global__ void __launch_bounds__(256) prefill_join_tail_kernel(const PrefillParams p) {
  constexpr int ROWS = D == 128 ? 256 : 128, STEPS = ROWS / 8;
  griddep_wait();
  for (int u = blockIdx.x;; u += gridDim.x) {
    const int tail = u / STEPS, r = u % STEPS * 8 + (threadIdx.x >> 5);
    const Share sh = find_share(p, tail, ROWS, true);
    if (sh.b < 0) return;   // past the last round's tiles (or there are none)
    const int flat = sh.first * ROWS + r;
    if (flat >= sh.len * p.G) continue;
    const size_t row = (size_t)(sh.start + flat / p.G) * p.Hq + sh.kvh * p.G + flat % p.G;
    join_row<D>(p, (size_t)tail * sh.pieces * ROWS + r, ROWS, sh.pieces, row, threadIdx.x & 31);
  }
}

}  // namespace pf
}  // namespace pa
