// pa_latent_decode.cu -- the absorbed form of latent attention over the paged cache:
// the split of the work, the choice of kernel, and the join of what was split.
#include "pa_latent_decode.cuh"

namespace pa {
namespace lat {
namespace {

// ----------------------------------------------------------------- the join

// W warps a row (four: a CTA each; one: four rows a CTA): zeros where there is no key, the
// joined pieces where a sequence's tiles went to several workers.  The first CTA joins the
// workers' flags too.  The first pieces are asked for together with the weights of all: the
// way from the starts to the output is three latencies long.
template <int W>
__global__ void __launch_bounds__(128) latent_join_kernel(const AbsorbedParams p) {
  constexpr int F = 4 / W, U = W == 4 ? 8 : 2;   // 16-byte parts of a row a thread; pieces of a sequence in flight
  const int tid = threadIdx.x, lane = tid & 31;
  const int all = p.Q * p.H, row = W == 4 ? blockIdx.x : blockIdx.x * 4 + (tid >> 5), b = row / all, r = row % all;
  const int grp = p.RG == 1 ? 0 : r / p.R, sets = p.RG / p.S, col = W == 4 ? tid : lane;
  griddep_launch();                     // (a call that follows may set itself up)
  griddep_wait();                       // the pieces are complete
  if (blockIdx.x == 0 && tid < 32) {
    uint32_t bits = 0;
    for (int i = lane; i < p.workers * p.S; i += 32) bits |= p.flags[i];
    bits = __reduce_or_sync(0xffffffffu, bits);
    if (lane == 0) p.hdr[HDR_ERR] = bits;
  }
  if (row >= p.B * all) return;
  const uint32_t start = p.starts[b], tiles = p.starts[b + 1] - start, last = p.starts[p.B];
  long long slot0 = 0;
  int parts = 0;
  bool skip = false;                    // of the first worker's slots
  if (tiles > 0) {
    const uint32_t run = run_of(p, last * sets), a = start * sets + (uint32_t)(grp / p.S) * tiles;
    const uint32_t c0 = a / run, c1 = (a + tiles - 1) / run;
    if (c0 == c1) return;               // written by the attention kernel
    parts = (int)(c1 - c0) + 1;
    slot0 = c0;
    skip = a != c0 * run;               // its piece is not the worker's first
  }
  auto at = [&](int k) {                // row of piece k among the partial ones
    return ((2 * (slot0 + k) + (k == 0 && skip ? 1 : 0)) * p.S + grp % p.S) * p.R + r % p.R;
  };
  float4 x[U][F];
  auto load = [&](int k0, int n) {
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int f = 0; f < F; ++f) {
        x[i][f] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < n) x[i][f] = __ldcs(reinterpret_cast<const float4 *>(p.part_o + at(k0 + i) * kLatent) + col + f * 32 * W);
      }
  };
  // every warp has the weights, 32 at a time, a lane each
  const float first = lane < parts ? p.part_lse[at(lane)] : kNegInf;
  load(0, parts);
  float M = first;
  for (int k = lane + 32; k < parts; k += 32) M = fmaxf(M, p.part_lse[at(k)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float sum = 0.f;
  float4 acc[F];
#pragma unroll
  for (int f = 0; f < F; ++f) acc[f] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < parts; k0 += 32) {
    const float ls = k0 == 0 ? first : k0 + lane < parts ? p.part_lse[at(k0 + lane)] : kNegInf;
    const float wl = ls == kNegInf ? 0.f : expf(ls - M);   // (a NaN among a piece's scores is in its lse)
    sum += wl;
    for (int j = 0; j < min(32, parts - k0); j += U) {
      if (k0 + j > 0) load(k0 + j, parts - k0 - j);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const float wt = __shfl_sync(0xffffffffu, wl, (j + i) & 31);
        if (wt == 0.f || k0 + j + i >= parts) continue;   // (a piece without keys)
#pragma unroll
        for (int f = 0; f < F; ++f) {
          acc[f].x += wt * x[i][f].x;
          acc[f].y += wt * x[i][f].y;
          acc[f].z += wt * x[i][f].z;
          acc[f].w += wt * x[i][f].w;
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll
  for (int f = 0; f < F; ++f) {
    const size_t to = (size_t)row * kLatent + 4 * (col + f * 32 * W);
    const float4 y = make_float4(acc[f].x * inv, acc[f].y * inv, acc[f].z * inv, acc[f].w * inv);
    if (p.out_fp32)
      *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + to) = y;
    else
      *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + to) =
          make_uint2(tc::f2_to_bf2(y.x, y.y), tc::f2_to_bf2(y.z, y.w));
  }
  if (col == 0 && p.lse_out) p.lse_out[row] = sum != 0.f ? M + logf(sum) : kNegInf;
}

}  // namespace

DecodePlan plan_latent_decode(int B, int Q, int H, int max_seq_len) {
  DecodePlan d;
  const int rows = Q * H, groups = (rows + kMaxRows - 1) / kMaxRows;
  d.RG = groups <= 8 ? groups : (groups + 7) / 8 * 8;
  d.S = groups <= 8 ? groups : 8;
  d.R = (rows + d.RG - 1) / d.RG;
  // one sequence of 1,000 keys, 20 heads: runs of 2, 3, 4, 6 or 8 tiles 13.5, 13.1, 12.8, 13.3 or
  // 13.9 us.  (Many short sequences pay for it: 64 of 32 keys, four to a worker, take 23 us.)
  d.least = 4;
  const long long tiles = (long long)B * (d.RG / d.S) * ((max_seq_len + 31LL) / 32), runs = (tiles + d.least - 1) / d.least;
  const long long most = kSms / d.S;
  d.workers = (int)(runs < 1 ? 1 : runs < most ? runs : most);
  return d;
}

cudaError_t launch_latent_decode(const AbsorbedParams &p, cudaStream_t s) {
  const cudaError_t e = launch_latent_rows(p, s);
  if (e != cudaSuccess) return e;
  // one warp a row where rows alone fill the GPU (64 sequences of 128 heads: 141 us with four
  // warps a row, 126 with one; 8 tokens of 24 heads of four: 124 with four, 134 with one)
  const int rows = p.B * p.Q * p.H;
  return rows <= 16 * kSms ? launch_pdl(latent_join_kernel<4>, (unsigned)rows, 128, 0, s, p)
                           : launch_pdl(latent_join_kernel<1>, (unsigned)((rows + 3) / 4), 128, 0, s, p);
}

}  // namespace lat
}  // namespace pa
