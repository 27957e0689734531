// pa_prefill.cu -- attention of a ragged batch of prompt chunks over the
// paged cache: causal, with the score options of pa_score.cuh.
//
// A row is one (query token, query head) of a kv head's group: row r of a
// sequence is token r / G, head r % G, so that the G heads that share a kv
// head share every key tile that is read.  Tiles of 64 rows walk the key
// tiles of 64 tokens that some row of theirs sees, with the running maximum
// and sum of the softmax per row.
#include "pa_launch.h"
#include "pa_score.cuh"

namespace pa {
namespace {

constexpr int kPfWarps = 4;
constexpr int kPfThreads = kPfWarps * 32;
constexpr int kPfRows = 16 * kPfWarps;
constexpr int kPfKeys = 64;

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&a)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&a)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// eight consecutive values of a cached row as bf16 (exact for every format:
// an int8 code, an E4M3 value and a product e2m1 * e4m3 have at most 8
// significant bits), without the int8 row scale and the per-tensor scales
template <int DT, int D>
__device__ __forceinline__ uint4 load8(const void *codes, const void *scales, size_t row, int chunk) {
  if constexpr (DT == PA_KV_BF16) {
    return __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(codes) + row * D * 2) + chunk);
  } else {
    float x[8];
    if constexpr (DT == PA_KV_INT8) {
      const uint2 u = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(codes) + row * D) + chunk);
      s8x4_to_f4(u.x, x);
      s8x4_to_f4(u.y, x + 4);
    } else if constexpr (DT == PA_KV_FP8) {
      const uint2 u = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(codes) + row * D) + chunk);
      const uint32_t w[4] = {u.x & 0xFFFFu, u.x >> 16, u.y & 0xFFFFu, u.y >> 16};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = h2u_to_f2(e4m3x2_u16_to_h2(w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    } else {
      const uint32_t u = __ldg(reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(codes) + row * (D / 2)) + chunk);
      const uint32_t sc = e4m3_to_h2_dup(__ldg(static_cast<const uint8_t *>(scales) + row * (D / 16) + (chunk >> 1)));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = h2u_to_f2(hmul2_u32(e2m1x2_to_h2((u >> (8 * i)) & 0xFFu), sc));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
    return make_uint4(bf2(x[0], x[1]), bf2(x[2], x[3]), bf2(x[4], x[5]), bf2(x[6], x[7]));
  }
}

// the sequence and row tile of tile index `tile` (tiles of all sequences in
// order, `per` tokens each): every thread of a warp gets the answer
struct TileOf {
  int b, first, start, len;   // sequence (-1: none), first token in it, its tokens' start, count
};
__device__ __forceinline__ TileOf find_tile(const PrefillParams &p, int tile, int rows_per_tile) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  uint32_t err = 0;
  TileOf r = {-1, 0, 0, 0};
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    int start = 0, len = 0;
    if (b < p.B) {
      const int s0 = __ldg(p.q_starts + b), s1 = __ldg(p.q_starts + b + 1);
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
      break;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (err) set_err(p.hdr, PA_ERRF_BAD_Q_START);
  return r;
}

template <int DT, int D>
__global__ void __launch_bounds__(kPfThreads) prefill_kernel(const PrefillParams p, int max_tiles) {
  constexpr int CH = D / 8;   // 16-byte chunks per row
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t *sQ = smem, *sK = sQ + kPfRows * D * 2, *sV = sK + kPfKeys * D * 2;
  __shared__ float s_ks[kPfKeys], s_vs[kPfKeys];
  __shared__ int s_ok[kPfKeys / kBlock];
  __shared__ int s_lo, s_hi, s_lo_max, s_hi_min;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int Hkv = p.kv.hkv, G = p.G;
  const int kvh = blockIdx.x % Hkv;
  const int rest = blockIdx.x / Hkv;
  const int split = rest % p.splits;
  const int tile = max_tiles - 1 - rest / p.splits;   // the last tokens see most: first
  const TileOf to = find_tile(p, tile, kPfRows);
  if (to.b < 0) return;
  const int b = to.b, row0 = to.first * kPfRows, nrows = min(kPfRows, to.len * G - row0);
  int n = __ldg(p.seq_lens + b);
  if (n < 0 || n > p.stride * kBlock || (n > 0 && n < to.len)) {
    if (tid == 0)
      set_err(p.hdr, n < 0 ? PA_ERRF_NEG_LEN : n < to.len ? PA_ERRF_LEN_LT_QLEN : PA_ERRF_LEN_OVER_CAPACITY);
    n = min(max(n, 0), p.stride * kBlock);
  }
  const int prefix = p.sc.prefix ? __ldg(p.sc.prefix + b) : 0;

  if (tid == 0) {
    s_lo = 0x7fffffff;
    s_hi = 0;
    s_lo_max = 0;
    s_hi_min = 0x7fffffff;
  }
  __syncthreads();
  // this thread's two rows
  int r_lo[2], r_hi[2], r_pos[2];
  float slope[2];
  size_t r_out[2];
  bool r_live[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = warp * 16 + (lane >> 2) + 8 * h;
    r_live[h] = r < nrows;
    const int rr = row0 + (r_live[h] ? r : 0);
    const int tok = rr / G, head = kvh * G + rr % G;
    r_pos[h] = n - to.len + tok;
    const int first = p.sc.first_key ? __ldg(p.sc.first_key + to.start + tok) : 0;
    KeyRange kr = key_range(p.sc, r_pos[h], n, first, prefix);
    r_out[h] = (size_t)(to.start + tok) * p.Hq + head;
    slope[h] = p.sc.slopes ? __ldg(p.sc.slopes + head) * 1.4426950408889634f : 0.f;
    if (!r_live[h]) kr.lo = kr.hi = 0;
    r_lo[h] = kr.lo;
    r_hi[h] = kr.hi;
    if (r_live[h]) {
      if (kr.hi > kr.lo) {
        atomicMin(&s_lo, kr.lo);
        atomicMax(&s_hi, kr.hi);
      }
      atomicMax(&s_lo_max, kr.lo);
      atomicMin(&s_hi_min, kr.hi);
    }
  }
  // queries
  for (int i = tid; i < kPfRows * CH; i += kPfThreads) {
    const int r = i / CH, c = i % CH;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (r < nrows) {
      const int rr = row0 + r;
      u = __ldg(reinterpret_cast<const uint4 *>(
                    p.q + ((size_t)(to.start + rr / G) * p.Hq + kvh * G + rr % G) * D) + c);
    }
    *reinterpret_cast<uint4 *>(sQ + r * D * 2 + ((c ^ (r & 7)) << 4)) = u;
  }
  __syncthreads();
  const int k_lo = s_lo < s_hi ? s_lo / kPfKeys : 0, k_hi = (s_hi + kPfKeys - 1) / kPfKeys;
  const int nt = max(0, k_hi - k_lo), per = (nt + p.splits - 1) / p.splits;
  const int t0 = k_lo + min(nt, split * per), t1 = k_lo + min(nt, (split + 1) * per);
  const int see_lo = s_lo, see_hi = s_hi;

  float o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
  float m[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f};
  const float kg = has_global_scale(DT) ? p.kv.kg : 1.f;
  const bool cap = p.sc.cap_log2 != 0.f;
  const float f = (cap ? p.sc.cap_in : p.scale_log2) * kg;
  const int *trow = p.tables + (size_t)b * p.stride;

  for (int kt = t0; kt < t1; ++kt) {
    __syncthreads();
    if (tid < kPfKeys / kBlock) {
      const int key = kt * kPfKeys + tid * kBlock;
      const int id = key < see_hi ? __ldg(trow + key / kBlock) : -1;
      const bool ok = id >= 0 && id < p.kv.num_blocks;
      if (key < see_hi && key + kBlock > see_lo && !ok) set_err(p.hdr, PA_ERRF_BAD_BLOCK_ID);
      s_ok[tid] = ok ? id : -1;
    }
    __syncthreads();
    for (int i = tid; i < kPfKeys * CH; i += kPfThreads) {
      const int r = i / CH, c = i % CH, key = kt * kPfKeys + r;
      uint4 k4 = make_uint4(0, 0, 0, 0), v4 = k4;
      const int id = s_ok[r / kBlock];
      float ks = 0.f, vs = 0.f;
      if (id >= 0 && key >= see_lo && key < see_hi) {
        const size_t row = ((size_t)id * Hkv + kvh) * kBlock + (key & (kBlock - 1));
        k4 = load8<DT, D>(p.kv.k, p.kv.ks, row, c);
        v4 = load8<DT, D>(p.kv.v, p.kv.vs, row, c);
        if constexpr (DT == PA_KV_INT8) {
          ks = fp16_bits_to_f(__ldg(static_cast<const uint16_t *>(p.kv.ks) + row));
          vs = fp16_bits_to_f(__ldg(static_cast<const uint16_t *>(p.kv.vs) + row));
        }
      }
      if (DT == PA_KV_INT8 && c == 0) {
        s_ks[r] = ks;
        s_vs[r] = vs;
      }
      const int off = r * D * 2 + ((c ^ (r & 7)) << 4);
      *reinterpret_cast<uint4 *>(sK + off) = k4;
      *reinterpret_cast<uint4 *>(sV + off) = v4;
    }
    __syncthreads();
    // S = Q K^T: 16 rows x 64 keys per warp
    float s[kPfKeys / 8][4];
#pragma unroll
    for (int i = 0; i < kPfKeys / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t a[4];
      {
        const int r = warp * 16 + (lane & 15), c = 2 * ks + (lane >> 4);
        ldsm4(smem_u32(sQ) + r * D * 2 + ((c ^ (r & 7)) << 4), a);
      }
#pragma unroll
      for (int nt2 = 0; nt2 < kPfKeys / 16; ++nt2) {
        uint32_t kb[4];
        const int r = nt2 * 16 + (lane & 7) + ((lane >> 4) << 3), c = 2 * ks + ((lane >> 3) & 1);
        ldsm4(smem_u32(sK) + r * D * 2 + ((c ^ (r & 7)) << 4), kb);
        mma_bf16(s[2 * nt2], a, kb[0], kb[1]);
        mma_bf16(s[2 * nt2 + 1], a, kb[2], kb[3]);
      }
    }
    // scores, masks
    float mx[2] = {m[0], m[1]};
#pragma unroll
    for (int i = 0; i < kPfKeys / 8; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int h = j >> 1, kk = i * 8 + 2 * (lane & 3) + (j & 1), key = kt * kPfKeys + kk;
        float x = s[i][j] * f;
        if constexpr (DT == PA_KV_INT8) x *= s_ks[kk];
        if (cap) x = capped(x, p.sc.cap_log2);
        x -= slope[h] * (float)abs(r_pos[h] - key);
        const bool see = key >= r_lo[h] && key < r_hi[h] && s_ok[kk / kBlock] >= 0;
        s[i][j] = see ? x : kNegInf;
        mx[h] = fmaxf(mx[h], s[i][j]);
      }
    }
    float al[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
      al[h] = mx[h] == kNegInf ? 1.f : score_ex2(m[h] - mx[h]);
      m[h] = mx[h];
      l[h] *= al[h];
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] *= al[j >> 1];
#pragma unroll
    for (int i = 0; i < kPfKeys / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int h = j >> 1;
        const float e = s[i][j] == kNegInf ? 0.f : score_ex2(s[i][j] - m[h]);
        l[h] += e;
        s[i][j] = DT == PA_KV_INT8 ? e * s_vs[i * 8 + 2 * (lane & 3) + (j & 1)] : e;
      }
    // O += P V
#pragma unroll
    for (int kk = 0; kk < kPfKeys / 16; ++kk) {
      const uint32_t a[4] = {bf2(s[2 * kk][0], s[2 * kk][1]), bf2(s[2 * kk][2], s[2 * kk][3]),
                             bf2(s[2 * kk + 1][0], s[2 * kk + 1][1]),
                             bf2(s[2 * kk + 1][2], s[2 * kk + 1][3])};
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        uint32_t vb[4];
        const int r = kk * 16 + (lane & 15), c = 2 * d + (lane >> 4);
        ldsm4_trans(smem_u32(sV) + r * D * 2 + ((c ^ (r & 7)) << 4), vb);
        mma_bf16(o[2 * d], a, vb[0], vb[1]);
        mma_bf16(o[2 * d + 1], a, vb[2], vb[3]);
      }
    }
  }
  const float vg = has_global_scale(DT) ? p.kv.vg : 1.f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    if (!r_live[h]) continue;
    const float inv = l[h] > 0.f ? vg / l[h] : 0.f;
    const float lse = l[h] > 0.f ? (m[h] + log2f(l[h])) * 0.69314718055994531f : kNegInf;
    if (p.splits > 1) {
      const size_t row = (size_t)split * p.T * p.Hq + r_out[h];
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<float2 *>(p.part_o + row * D + i * 8 + 2 * (lane & 3)) =
            make_float2(o[i][2 * h] * inv, o[i][2 * h + 1] * inv);
      if ((lane & 3) == 0) p.part_lse[row] = lse;
      continue;
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      const size_t at = r_out[h] * D + i * 8 + 2 * (lane & 3);
      const float x = o[i][2 * h] * inv, y = o[i][2 * h + 1] * inv;
      if (p.out_fp32)
        *reinterpret_cast<float2 *>(static_cast<float *>(p.out) + at) = make_float2(x, y);
      else
        *reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(p.out) + at) = bf2(x, y);
    }
    if ((lane & 3) == 0 && p.lse_out) p.lse_out[r_out[h]] = lse;
  }
}

// joins the key splits of every row of the batch's sequences: one warp a row
template <int D>
__global__ void __launch_bounds__(256) prefill_join_kernel(const PrefillParams p) {
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
          make_uint2(bf2(x[0], x[1]), bf2(x[2], x[3]));
  }
  if (lane == 0 && p.lse_out) p.lse_out[row] = sum > 0.f ? M + logf(sum) : kNegInf;
}

template <int DT, int D>
cudaError_t launch_one(const PrefillParams &p, cudaStream_t s) {
  constexpr int smem = (kPfRows + 2 * kPfKeys) * D * 2;
  auto kern = prefill_kernel<DT, D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  // every sequence has at most one tile that is not full
  const long long tiles = (long long)p.T * p.G / kPfRows + p.B;
  const long long grid = tiles * p.kv.hkv * p.splits;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  kern<<<(unsigned)grid, kPfThreads, smem, s>>>(p, (int)tiles);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.splits == 1) return e;
  const long long rows = (long long)p.T * p.Hq;
  prefill_join_kernel<D><<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

// key splits per row tile: one unless the row tiles leave half of the SMs idle
int prefill_splits(int T, int B, int Hkv, int G, int D, int max_seq_len) {
  (void)D;
  const long long ctas = ((long long)T * G / kPfRows + B) * Hkv;
  const long long most = (max_seq_len + 4 * kPfKeys - 1) / (4 * kPfKeys);   // at least 256 keys each
  long long s = 304 / (ctas > 0 ? ctas : 1);
  s = s < most ? s : most;
  return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}

cudaError_t launch_prefill(const PrefillParams &p, cudaStream_t s) {
  switch (p.kv.dtype * 2 + (p.kv.D == 256)) {
    case PA_KV_BF16 * 2: return launch_one<PA_KV_BF16, 128>(p, s);
    case PA_KV_BF16 * 2 + 1: return launch_one<PA_KV_BF16, 256>(p, s);
    case PA_KV_INT8 * 2: return launch_one<PA_KV_INT8, 128>(p, s);
    case PA_KV_INT8 * 2 + 1: return launch_one<PA_KV_INT8, 256>(p, s);
    case PA_KV_NVFP4 * 2: return launch_one<PA_KV_NVFP4, 128>(p, s);
    case PA_KV_NVFP4 * 2 + 1: return launch_one<PA_KV_NVFP4, 256>(p, s);
    case PA_KV_FP8 * 2: return launch_one<PA_KV_FP8, 128>(p, s);
    case PA_KV_FP8 * 2 + 1: return launch_one<PA_KV_FP8, 256>(p, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace pa
