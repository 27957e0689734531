// pa_latent_decode.cuh -- the parts of the absorbed form: a worker's run of key tiles and
// its pieces, conversion of FP8 rows, the write of the output, the tensor maps.
#pragma once

#include "pa_latent_umma.cuh"

namespace pa {
namespace lat {

constexpr int kMaxStages = 5;

// Weights are relative to a row's maximum over its piece's first tile, whatever follows
// (no maximum to agree on, no output to rescale, in any tile); where they sum to more
// than this in a thread and tile, the worker goes over its run again, each piece twice:
// for its maximum, then for its output.  fp16 weights hold 2^15, bf16 and fp32 2^127.
// One row of a run is enough.  64 sequences of 128 heads, a late key of each 18 (FP8) or 34
// nats (bf16) above the others for one head: 318 us instead of 127, 248 instead of 105.
template <bool FP8>
constexpr float kMost = FP8 ? 0x1p13f : 0x1p32f;

// What every role knows of the worker's run: where it starts, its tiles, and the keys
// of its first sequence.
struct Run {
  int b, set, tile, count, n;
  int sums[32];
};

__device__ __forceinline__ int keys_of(const AbsorbedParams &p, int b) {
  const int capacity = (int)min((long long)p.stride * kBlock, 0x7fffffffLL);
  return min(max(__ldg(p.seq_lens + b), 0), capacity);
}
template <int TK>
__device__ __forceinline__ int tiles_of(int n) { return n / TK + (n % TK != 0); }
// Tiles a worker takes.  (All of them are fewer than 2^31: the host sees to it.)
__device__ __forceinline__ uint32_t run_of(const AbsorbedParams &p, uint32_t total) {
  const uint32_t w = (uint32_t)p.workers;
  return max(total / w + (total % w != 0), (uint32_t)p.least);
}

// The pieces of a worker's run, one sequence (and set of groups) each.
template <int TK>
struct Piece {
  int b, set, t0, t1, tiles, n, left;   // tiles [t0, t1) of `tiles`; n keys; tiles left after
  bool first;
  __device__ __forceinline__ Piece(const Run &c)
      : b(c.b), set(c.set), t0(0), t1(c.tile), tiles(0), n(c.n), left(c.count), first(true) {}
  __device__ __forceinline__ bool next(const AbsorbedParams &p) {
    if (left <= 0) return false;
    if (tiles == 0) {                   // the first one: starts at t1
      t0 = t1;
      tiles = tiles_of<TK>(n);
    } else {
      first = false;
      t0 = 0;
      if (p.RG == p.S || ++set == p.RG / p.S) {
        set = 0;
        n = keys_of(p, ++b);
        while ((tiles = tiles_of<TK>(n)) == 0) n = keys_of(p, ++b);   // (some sequence follows: tiles are left)
      }
    }
    const int cnt = min(tiles - t0, left);
    t1 = t0 + cnt;
    left -= cnt;
    return true;
  }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
};

// Finds the worker's run: every thread sums the tiles of its share of the
// sequences, a scan over the CTA gives what is before them.  The first CTA also
// writes the sums for the join, and the flags of the lengths.
template <int TK>
__device__ __forceinline__ void find_run(const AbsorbedParams &p, Run &c, uint32_t *flags, int worker, bool head) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  const int per = p.B <= (int)blockDim.x ? 1 : (p.B + blockDim.x - 1) / blockDim.x;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  int sum = 0, n0 = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = keys_of(p, b);
    if (b == b0) n0 = n;
    sum += tiles_of<TK>(n);
    if (head) {
      const int x = __ldg(p.seq_lens + b);
      if (x != 0 && x < p.Q) set_err(flags, x < 0 ? PA_ERRF_NEG_LEN : PA_ERRF_LEN_LT_QLEN);
      if (x > (long long)p.stride * kBlock) set_err(flags, PA_ERRF_LEN_OVER_CAPACITY);
    }
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) c.sums[warp] = inc;
  if (tid == 0) c.count = 0;
  __syncthreads();
  uint32_t before = inc - sum, all = 0;
  for (int w = 0; w < nw; ++w) {
    const uint32_t x = c.sums[w];
    if (w < warp) before += x;
    all += x;
  }
  const uint32_t sets = p.RG == p.S ? 1 : p.RG / p.S;
  const uint32_t total = all * sets, run = run_of(p, total);
  const uint32_t x0 = min(total, run * worker), x1 = min(total, x0 + run);
  if (head) {
    int a = before;
    for (int b = b0; b < b1; ++b) {
      p.starts[b] = a;
      a += tiles_of<TK>(keys_of(p, b));
    }
    if (tid == 0) p.starts[p.B] = all;
  }
  // the thread whose sequences hold tile x0
  uint32_t at = before * sets;
  if (x0 < x1 && at <= x0 && x0 < at + sum * sets) {
    int b = b0, n = n0;
    uint32_t t = tiles_of<TK>(n);
    while (x0 >= at + t * sets) {
      at += t * sets;
      n = keys_of(p, ++b);
      t = tiles_of<TK>(n);
    }
    c.b = b;
    c.set = sets == 1 ? 0 : (x0 - at) / t;
    c.tile = (x0 - at) - c.set * t;
    c.n = n;
    c.count = (int)(x1 - x0);
  }
  __syncthreads();
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// O^T (four blocks of 128 dims, a dim a lane, N columns each from `col` on) times a
// row's factor, to the rows of the output or of a piece.  A factor of 0: zeros, whatever
// O is.  The loops hold no branch on a row: with two a value 64 rows took 13,000 cycles.
template <int N>
__device__ __forceinline__ void write_rows(const AbsorbedParams &p, uint32_t col, const float *fac, int rows, bool whole,
                                           long long r_out, long long slot, int w, int lane) {
  constexpr int C = N < 32 ? N : 32;
  auto each = [&](auto *const base) {
#pragma unroll 1
    for (int r0 = 0; r0 < N && r0 < rows; r0 += C) {
      float inv[C];
#pragma unroll
      for (int i = 0; i < C; i += 4) {
        const float4 f = *reinterpret_cast<const float4 *>(fac + r0 + i);
        inv[i] = f.x;
        inv[i + 1] = f.y;
        inv[i + 2] = f.z;
        inv[i + 3] = f.w;
      }
#pragma unroll 1
      for (int mb = 0; mb < 4; ++mb) {
        float o[C];
        if constexpr (C == 32) {
          pf::ld32_issue(col + mb * N + r0, o);
          pf::ld_wait(o);
        } else {
          tmem_ld16(col + mb * N + r0, o);
        }
        auto *const to = base + (size_t)r0 * kLatent + mb * 128;
#pragma unroll
        for (int i = 0; i < C; ++i) o[i] = inv[i] != 0.f ? o[i] * inv[i] : 0.f;
        auto put = [&](int i) {
          if constexpr (sizeof(*base) == 4) to[i * kLatent] = o[i];
          else to[i * kLatent] = __float2bfloat16_rn(o[i]);
        };
        if (r0 + C <= rows) {
#pragma unroll
          for (int i = 0; i < C; ++i) put(i);
        } else {
#pragma unroll
          for (int i = 0; i < C; ++i)
            if (r0 + i < rows) put(i);
        }
      }
    }
  };
  const size_t at = (size_t)w * 32 + lane;
  if (!whole) each(p.part_o + slot * kLatent + at);
  else if (p.out_fp32) each(static_cast<float *>(p.out) + r_out * kLatent + at);
  else each(static_cast<__nv_bfloat16 *>(p.out) + r_out * kLatent + at);
}

template <typename P>
__device__ __forceinline__ long long group_row(const AbsorbedParams &p, const P &x, int sub, int &rows) {
  const int grp = x.set * p.S + sub, all = p.Q * p.H;
  rows = max(0, min(p.R, all - grp * p.R));
  return (long long)x.b * all + (long long)grp * p.R;
}

// sixteen E4M3 codes -> f16, exact
__device__ __forceinline__ void e4m3x16(const uint4 &u, uint32_t (&h)[8]) {
  const uint32_t word[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    h[2 * k] = e4m3x2_u16_to_h2(word[k] & 0xFFFFu);
    h[2 * k + 1] = e4m3x2_u16_to_h2(word[k] >> 16);
  }
}
// eight bf16 -> f16 (exact in its normal range)
__device__ __forceinline__ uint4 bf16x8_to_h(const uint4 &u) {
  const float2 a = bf16x2_to_f2(u.x), b = bf16x2_to_f2(u.y), d = bf16x2_to_f2(u.z), e = bf16x2_to_f2(u.w);
  return make_uint4(tc::f2_to_h2(a.x, a.y), tc::f2_to_h2(b.x, b.y), tc::f2_to_h2(d.x, d.y), tc::f2_to_h2(e.x, e.y));
}

// the cache in pages as [2 row groups][8 chunks of 64 dims][8 rows][64 dims], a page a copy,
// and its rotated parts
inline bool cache_maps(const AbsorbedParams &p, CUtensorMap *mc, CUtensorMap *mr) {
  const uint64_t nb = (uint64_t)p.kv.num_blocks;
  const uint64_t dc[4] = {64, 8, 8, nb * 2}, sc[3] = {kLatent * 2, 128, 8 * kLatent * 2};
  const uint32_t bc[4] = {64, 8, 8, 2};
  const uint64_t dr[2] = {kRope, nb * kBlock}, sr[1] = {kRope * 2};
  const uint32_t br[2] = {kRope, kBlock};
  return make_map(mc, p.kv.latent, 4, dc, sc, bc) && make_map(mr, p.kv.rope, 2, dr, sr, br);
}
// the queries' rows as [9 chunks of 64 dims][rows][64 dims], all chunks of `rows` rows a copy
inline bool query_map(const AbsorbedParams &p, CUtensorMap *mq, uint32_t rows) {
  const uint64_t dims[3] = {64, (uint64_t)p.B * p.Q * p.H, 9}, strides[2] = {kRow * 2, 128};
  const uint32_t box[3] = {64, rows, 9};
  return make_map(mq, p.q, 3, dims, strides, box);
}

cudaError_t launch_latent_rows(const AbsorbedParams &p, cudaStream_t s);

}  // namespace lat
}  // namespace pa
