// pa_latent_decode.cu -- the absorbed form of latent attention over the paged
// cache on the 5th-generation tensor cores (tcgen05.mma, accumulators in tensor
// memory).
//
// A row is one (token, head) of a sequence; the R <= 64 rows of a group share
// every key.  Per tile of 64 keys, in fp32 accumulation:
//   S [64 rows x 64 keys] = Q [64 x 576] . K^T     both K-major in shared memory
//   P = exp2(S * scale - m)                        to shared memory, 16 bits
//   O^T [512 x N] += C^T [512 x 64] . P^T [64 x N] A = the same tile, MN-major
// A cached row is key and value at once, so a tile is brought in once and read by
// both products as it lies.  With the latent dims on the instruction's M side the
// output takes 4 N columns of tensor memory (N = 16, 32 or 64 rows) instead of 512.
// The running maximum moves only when a score passes it by 2^8.  P is rounded
// once, to bf16 (bf16 cache) or fp16.
//
// A 16-token page lies in shared memory as [2 row groups][8 chunks of 64 dims][8
// rows][128 bytes], swizzled: one four-dimensional tiled copy a page (and one of its
// rotated part), its eight-row groups a uniform 8 KB apart for both majors.
//
// Work: see DecodePlan.  A run of tiles may start and end inside a sequence; the
// pieces of a sequence that several workers share are joined by their log-sum-exp
// in a second kernel.
//
// Roles: four softmax warps (16 rows each; they also write the output), a warp for
// each product, one that copies pages, others for the queries and, FP8, for turning
// codes into f16 (exact).  Hand-offs are mbarriers; waits are capped.
#include "pa_latent_umma.cuh"

namespace pa {
namespace lat {
namespace {

constexpr float kLazy = 8.0f;                     // log2 of how far a score may pass the running maximum
constexpr int kMaxStages = 5;
constexpr int kWide = 32;
constexpr uint32_t kColS = 0, kColO = 128;        // two S buffers, O^T of 4 N columns
constexpr uint32_t kBarSoft = 1;                  // named barrier of the softmax warps

template <bool FP8, int N>
struct Geo {
  static constexpr int TK = N == 64 ? kWide : 32, PG = TK / kBlock;
  static constexpr uint32_t QCHUNK = N * 128, QBYTES = 9 * QCHUNK;   // [N rows][128 bytes] a chunk of 64 dims
  static constexpr uint32_t LAT = TK * kLatent * 2, STAGE = LAT + TK * kRope * 2;
  static constexpr int PB = TK == 32 ? 2 : 1;                        // P buffers: halves of its 128-byte rows
  static constexpr int FIT = (227 * 1024 - 3072 - QBYTES - QCHUNK) / STAGE;
  static constexpr int NS = FIT < kMaxStages ? FIT : kMaxStages;
  static constexpr int QWARPS = FP8 ? 4 : 1, FWARPS = FP8 ? 8 : 1;   // queries; pages
  static constexpr int WARP_S = 4, WARP_O = 5, WARP_Q = 6, WARP_F = WARP_Q + QWARPS;
  static constexpr int THREADS = (WARP_F + FWARPS + 3) / 4 * 128;
  static constexpr uint32_t OFF_K = QBYTES, OFF_P = OFF_K + NS * STAGE;
  static constexpr uint32_t SMEM = OFF_P + QCHUNK + 1024;
  static_assert(SMEM + 2048 <= 227 * 1024, "shared memory (with the static control block)");
};

struct Ctl {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t sfull[2], pready[2], odone[2], qfull, qfree, done;   // (of even and odd tiles)
  uint32_t tmem;
  int abort;
  int b, set, tile, count;              // where the worker's run starts; its tiles
  int sums[32];
  uint32_t dead[kMaxStages];            // bit j: page j of the tile has a bad id
  float fac[kMaxRows];                  // a row's rescale, at the end its 1 / sum
};
static_assert(sizeof(Ctl) <= 2048, "Geo::SMEM leaves 2 KB");

__device__ __forceinline__ int keys_of(const AbsorbedParams &p, int b) {
  const int capacity = (int)min((long long)p.stride * kBlock, 0x7fffffffLL);
  return min(max(__ldg(p.seq_lens + b), 0), capacity);
}
template <int TK>
__device__ __forceinline__ int tiles_of(int n) { return (n + TK - 1) / TK; }
// tiles a worker takes
__device__ __forceinline__ long long run_of(const AbsorbedParams &p, long long total) {
  return (total + p.workers - 1) / p.workers;
}

// The pieces of a worker's run, one sequence (and set of groups) each.
template <int TK>
struct Piece {
  int b, set, t0, t1, tiles, n, left;   // tiles [t0, t1) of `tiles`; n keys; tiles left after
  bool first;
  __device__ __forceinline__ Piece(const Ctl &c) : b(c.b), set(c.set), t0(0), t1(c.tile), tiles(0), n(0), left(c.count), first(true) {}
  __device__ __forceinline__ bool next(const AbsorbedParams &p) {
    if (left <= 0) return false;
    if (tiles == 0) {                   // the first one: starts at t1
      t0 = t1;
    } else {
      first = false;
      t0 = 0;
      if (++set == p.RG / p.S) {
        set = 0;
        ++b;
      }
    }
    n = keys_of(p, b);
    while ((tiles = tiles_of<TK>(n)) == 0) n = keys_of(p, ++b);   // (some sequence follows: tiles are left)
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
__device__ __forceinline__ void find_run(const AbsorbedParams &p, Ctl &c, int worker, bool head) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  const int per = (p.B + blockDim.x - 1) / blockDim.x;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  int sum = 0;
  for (int b = b0; b < b1; ++b) {
    sum += tiles_of<TK>(keys_of(p, b));
    if (head) {
      const int n = __ldg(p.seq_lens + b);
      if (n != 0 && n < p.Q) flag(p.hdr, n < 0 ? PA_ERRF_NEG_LEN : PA_ERRF_LEN_LT_QLEN);
      if (n > (long long)p.stride * kBlock) flag(p.hdr, PA_ERRF_LEN_OVER_CAPACITY);
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
  int before = inc - sum, all = 0;
  for (int w = 0; w < nw; ++w) {
    if (w < warp) before += c.sums[w];
    all += c.sums[w];
  }
  const int sets = p.RG / p.S;
  const long long total = (long long)all * sets, run = run_of(p, total);
  const long long x0 = run * worker, x1 = min(total, x0 + run);
  if (head) {
    int a = before;
    for (int b = b0; b < b1; ++b) {
      p.starts[b] = a;
      a += tiles_of<TK>(keys_of(p, b));
    }
    if (tid == 0) p.starts[p.B] = all;
  }
  // the thread whose sequences hold tile x0
  long long at = (long long)before * sets;
  if (x0 < x1 && at <= x0 && x0 < at + (long long)sum * sets) {
    int b = b0, t;
    for (;; ++b) {
      t = tiles_of<TK>(keys_of(p, b));
      if (x0 < at + (long long)t * sets) break;
      at += (long long)t * sets;
    }
    c.b = b;
    c.set = (int)((x0 - at) / t);
    c.tile = (int)((x0 - at) % t);
    c.count = (int)(x1 - x0);
  }
  __syncthreads();
}

// ------------------------------------------------------------------- products

// A warp for each product: between a commit and the next product of the same warp
// lie some 350 cycles of barrier latencies, which pass under the other's products.
// (One warp for both, whichever could go: 2,180 cycles for 32 keys of 64 rows, of
// which the products take 1,280; a verify step of 192 rows at 64K keys 174 us.)
// S of a tile waits for its copy and for the weights of the tile before last, whose
// buffer it takes.
template <bool FP8, int N>
__device__ void role_scores(const AbsorbedParams &p, uint8_t *smem, Ctl &c, uint32_t tmem) {
  using G = Geo<FP8, N>;
  constexpr uint32_t IQK = idesc_of(!FP8, 64, G::TK, false, false);
  const uint32_t lead = elect_one();
  const uint64_t dQ = sdesc(smem_u32(smem), 16, 1024);
  const uint64_t dK = sdesc(smem_u32(smem + G::OFF_K), 16, 8192);
  const uint64_t dR = sdesc(smem_u32(smem + G::OFF_K + G::LAT), 16, 1024);
  uint32_t g = 0, piece = 0;
  Piece<G::TK> x(c);
  for (; x.next(p); ++piece) {
    wait_cap(&c.qfull, piece & 1, &c.abort, p.hdr);
#pragma unroll 1
    for (int t = x.t0; t < x.t1; ++t, ++g) {
      const uint32_t st = g % G::NS;
      if (g >= 2) wait_cap(&c.pready[g & 1], ((g >> 1) - 1) & 1, &c.abort, p.hdr);
      wait_cap(&c.full[st], (g / G::NS) & 1, &c.abort, p.hdr);
      tc_fence_after();
      const uint64_t at = (uint64_t)(st * (G::STAGE >> 4));
      const uint32_t d = tmem + kColS + (g & 1) * G::TK;
#pragma unroll
      for (int ch = 0; ch < 8; ++ch)
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_ss_if(lead, d, dQ + (uint64_t)((ch * G::QCHUNK + ks * 32) >> 4),
                    dK + at + (uint64_t)((ch * 1024 + ks * 32) >> 4), IQK, ch + ks > 0 ? 1u : 0u);
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        mma_ss_if(lead, d, dQ + (uint64_t)((8 * G::QCHUNK + ks * 32) >> 4), dR + at + (uint64_t)((ks * 32) >> 4), IQK, 1u);
      commit_if(lead, &c.sfull[g & 1]);
      if (t + 1 == x.t1) commit_if(lead, &c.qfree);
    }
  }
  commit_if(lead, &c.done);   // tensor memory is released only after every product completes
  drain_wait(&c.done, 0);
  __syncwarp();
}

template <bool FP8, int N>
__device__ void role_output(const AbsorbedParams &p, uint8_t *smem, Ctl &c, uint32_t tmem) {
  using G = Geo<FP8, N>;
  constexpr uint32_t IPV = idesc_of(!FP8, 128, N, true, false);
  const uint32_t lead = elect_one();
  const uint64_t dC = sdesc(smem_u32(smem + G::OFF_K), 1024, 8192);
  const uint64_t dP = sdesc(smem_u32(smem + G::OFF_P), 16, 1024);
  uint32_t g = 0;
  Piece<G::TK> x(c);
  while (x.next(p)) {
#pragma unroll 1
    for (int t = x.t0; t < x.t1; ++t, ++g) {
      const uint32_t st = g % G::NS;
      wait_cap(&c.full[st], (g / G::NS) & 1, &c.abort, p.hdr);
      wait_cap(&c.pready[g & 1], (g >> 1) & 1, &c.abort, p.hdr);
      tc_fence_after();
      const uint64_t at = (uint64_t)(st * (G::STAGE >> 4));
      const uint64_t pb = dP + (uint64_t)((g % G::PB) * 64 >> 4);
#pragma unroll
      for (int ks = 0; ks < G::PG; ++ks)
#pragma unroll
        for (int mb = 0; mb < 4; ++mb)
          mma_ss_if(lead, tmem + kColO + mb * N, dC + at + (uint64_t)((ks * 16384 + mb * 2048) >> 4),
                    pb + (uint64_t)((ks * 32) >> 4), IPV, t > x.t0 || ks > 0 ? 1u : 0u);
      commit_if(lead, &c.empty[st]);
      commit_if(lead, &c.odone[g & 1]);
    }
  }
  commit_if(lead, &c.done);
  drain_wait(&c.done, 0);
  __syncwarp();
}

// -------------------------------------------------------------- copies (bf16)

// lane j < PG copies page j of every tile
template <int N>
__device__ __forceinline__ void role_copy(const AbsorbedParams &p, const CUtensorMap *mc, const CUtensorMap *mr,
                                          uint8_t *stages, Ctl &c) {
  using G = Geo<false, N>;
  const int lane = threadIdx.x & 31;
  uint32_t g = 0;
  bool ok = true;
  Piece<G::TK> x(c);
  while (ok && x.next(p)) {
    const int *row = p.tables + (size_t)x.b * p.stride;
#pragma unroll 1
    for (int t = x.t0; t < x.t1; ++t, ++g) {
      const uint32_t st = g % G::NS;
      const int key = t * G::TK + lane * kBlock;
      const bool in = lane < G::PG && key < x.n;
      const int id = in ? __ldg(row + key / kBlock) : 0;
      const bool bad = in && (uint32_t)id >= (uint32_t)p.kv.num_blocks;
      const uint32_t dead = __ballot_sync(0xffffffffu, bad);
      if (g >= G::NS) ok = wait_cap(&c.empty[st], (g / G::NS - 1) & 1, &c.abort, p.hdr);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (dead && lane == 0) flag(p.hdr, PA_ERRF_BAD_BLOCK_ID);
      if (lane < G::PG) {
        if (lane == 0) c.dead[st] = dead;
        if (in && !bad) {
          mbar_arrive_expect_tx(&c.full[st], kBlock * kRow * 2);
          const uint32_t dst = smem_u32(stages + st * G::STAGE);
          tma_4d(dst + lane * 16384, mc, 0, 0, 0, id * 2, &c.full[st]);
          tma_2d(dst + G::LAT + lane * 2048, mr, 0, id * kBlock, &c.full[st]);
        } else {
          mbar_arrive(&c.full[st]);
        }
      }
    }
  }
  // nothing lands after the CTA's end: the last fill of each stage
  for (uint32_t k = g > G::NS ? g - G::NS : 0; k < g; ++k) drain_wait(&c.full[k % G::NS], (k / G::NS) & 1);
  __syncwarp();
}

// ------------------------------------------------- FP8: codes to f16 (exact)

// 256 threads, 32 lanes a key row (16 codes each), eight rows apart; then the
// rotated parts, eight lanes a row.  The next tile's codes are requested before the
// present one's are converted.
template <int N>
__device__ __forceinline__ void role_dequant(const AbsorbedParams &p, uint8_t *stages, Ctl &c, int t) {
  using G = Geo<true, N>;
  constexpr int RI = G::TK / 8, RR = G::TK / 32;   // rows of codes, pieces of rotated parts a thread
  const int lane = t & 31, w = t >> 5;
  struct Raw {
    uint4 code[RI], rr[RR];
    uint32_t dead;
  };
  auto load = [&](const Piece<G::TK> &x, int tile, Raw &v) {
    const int *row = p.tables + (size_t)x.b * p.stride;
    const int k0 = tile * G::TK;
    int id[G::PG];
    v.dead = 0;
#pragma unroll
    for (int j = 0; j < G::PG; ++j) {
      const int key = k0 + j * kBlock;
      id[j] = key < x.n ? __ldg(row + key / kBlock) : -1;
      if ((uint32_t)id[j] >= (uint32_t)p.kv.num_blocks) {
        if (key < x.n) v.dead |= 1u << j;
        id[j] = -1;
      }
    }
#pragma unroll
    for (int i = 0; i < RI; ++i) {   // row w + 8 i, in page i / 2
      v.code[i] = make_uint4(0, 0, 0, 0);
      if (id[i >> 1] >= 0)
        v.code[i] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.kv.latent) +
                                                          ((size_t)id[i >> 1] * kBlock + (i & 1) * 8 + w) * kLatent) + lane);
    }
#pragma unroll
    for (int i = 0; i < RR; ++i) {   // row t / 8 + 32 i
      const int pg = t < 128 ? id[2 * i] : id[2 * i + 1];
      v.rr[i] = make_uint4(0, 0, 0, 0);
      if (pg >= 0)
        v.rr[i] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.kv.rope) +
                                                        ((size_t)pg * kBlock + ((t >> 3) & 15)) * kRope) + (t & 7));
    }
  };
  uint32_t g = 0;
  Piece<G::TK> x(c);
  Raw raw;
  bool more = x.next(p);
  int tile = x.t0;
  if (more) load(x, tile, raw);
  while (more) {
    const Raw v = raw;
    if (++tile == x.t1) {
      more = x.next(p);
      tile = x.t0;
    }
    if (more) load(x, tile, raw);
    const uint32_t st = g % G::NS;
    if (g >= G::NS) wait_cap(&c.empty[st], (g / G::NS - 1) & 1, &c.abort, p.hdr);
    const uint32_t dst = smem_u32(stages + st * G::STAGE);
    // the row's place in its group of eight is w: group i, chunk lane / 4
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      const uint32_t word[4] = {v.code[i].x, v.code[i].y, v.code[i].z, v.code[i].w};
      uint32_t h[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        h[2 * k] = e4m3x2_u16_to_h2(word[k] & 0xFFFFu);
        h[2 * k + 1] = e4m3x2_u16_to_h2(word[k] >> 16);
      }
      const uint32_t at = dst + i * 8192 + (lane >> 2) * 1024 + w * 128;
      const uint32_t p0 = 2 * (lane & 3);
      sts_u4(at + ((p0 ^ w) << 4), h[0], h[1], h[2], h[3]);
      sts_u4(at + (((p0 + 1) ^ w) << 4), h[4], h[5], h[6], h[7]);
    }
#pragma unroll
    for (int i = 0; i < RR; ++i) {
      const int r = (t >> 3) + 32 * i;
      const float2 a = bf16x2_to_f2(v.rr[i].x), b = bf16x2_to_f2(v.rr[i].y), d = bf16x2_to_f2(v.rr[i].z),
                   e = bf16x2_to_f2(v.rr[i].w);
      sts_u4(dst + G::LAT + r * 128 + (((t & 7) ^ (r & 7)) << 4), tc::f2_to_h2(a.x, a.y), tc::f2_to_h2(b.x, b.y),
             tc::f2_to_h2(d.x, d.y), tc::f2_to_h2(e.x, e.y));
    }
    if (t == 0) {
      c.dead[st] = v.dead;
      if (v.dead) flag(p.hdr, PA_ERRF_BAD_BLOCK_ID);
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.full[st]);
    ++g;
  }
}

// -------------------------------------------------------------------- queries

template <typename P>
__device__ __forceinline__ long long group_row(const AbsorbedParams &p, const P &x, int sub, int &rows) {
  const int grp = x.set * p.S + sub, all = p.Q * p.H;
  rows = max(0, min(p.R, all - grp * p.R));
  return (long long)x.b * all + (long long)grp * p.R;
}

template <bool FP8, int N>
__device__ __forceinline__ void role_query(const AbsorbedParams &p, const CUtensorMap *mq, uint8_t *smem, Ctl &c,
                                           int sub, int t) {
  using G = Geo<FP8, N>;
  uint32_t piece = 0;
  Piece<G::TK> x(c);
  while (x.next(p)) {
    if (piece > 0 && !wait_cap(&c.qfree, (piece - 1) & 1, &c.abort, p.hdr)) break;
    int rows;
    const long long r0 = group_row(p, x, sub, rows);
    if constexpr (!FP8) {
      if (t == 0) {
        mbar_arrive_expect_tx(&c.qfull, 9 * N * 128);
#pragma unroll 1
        for (int ch = 0; ch < 9; ++ch) tma_2d(smem_u32(smem + ch * G::QCHUNK), mq, ch * 64, (int)r0, &c.qfull);
      }
    } else {   // f16 (exact in its normal range); rows past the group are zeros
      constexpr int PIECES = N * 72, BATCH = 9;
#pragma unroll 1
      for (int i0 = t; i0 < PIECES; i0 += 128 * BATCH) {
        uint4 v[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
          const int i = i0 + k * 128, r = i / 72;
          v[k] = make_uint4(0, 0, 0, 0);
          if (i < PIECES && r < rows) v[k] = __ldg(reinterpret_cast<const uint4 *>(p.q + (r0 + r) * kRow) + i % 72);
        }
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
          const int i = i0 + k * 128, r = i / 72, ch = (i % 72) >> 3, q = i & 7;   // (72 is a multiple of 8)
          if (i >= PIECES) break;
          const float2 a = bf16x2_to_f2(v[k].x), b = bf16x2_to_f2(v[k].y), d = bf16x2_to_f2(v[k].z),
                       e = bf16x2_to_f2(v[k].w);
          sts_u4(smem_u32(smem + ch * G::QCHUNK) + r * 128 + ((q ^ (r & 7)) << 4), tc::f2_to_h2(a.x, a.y),
                 tc::f2_to_h2(b.x, b.y), tc::f2_to_h2(d.x, d.y), tc::f2_to_h2(e.x, e.y));
        }
      }
      fence_async_smem();
      __syncwarp();
      if ((t & 31) == 0) mbar_arrive(&c.qfull);
    }
    ++piece;
  }
  if constexpr (!FP8)
    if (t == 0 && piece > 0) drain_wait(&c.qfull, (piece - 1) & 1);
  __syncwarp();
}

// -------------------------------------------------------------------- softmax

template <bool FP8, int N>
__device__ void role_softmax(const AbsorbedParams &p, uint8_t *smem, Ctl &c, uint32_t tmem, int worker, int sub) {
  using G = Geo<FP8, N>;
  constexpr int TK = G::TK, NV = TK / 2;   // scores a thread
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, qd = lane & 3;
  const bool act = w * 16 < N;             // this warp has rows of S
  const int row0 = w * 16 + (lane >> 2);   // and row0 + 8
  const uint32_t lane_off = (uint32_t)(w * 32) << 16;
  const uint32_t sP = smem_u32(smem + G::OFF_P);
  const float f = p.scale_log2 * p.kv.g;
  uint32_t g = 0;
  Piece<G::TK> x(c);
  while (x.next(p)) {
    int rows;
    const long long r_out = group_row(p, x, sub, rows);
    const int first_row = (x.set * p.S + sub) * p.R;
    // keys that this thread's rows see (rows past the group: all), and the least of the group
    auto sees = [&](int r) { return r < rows ? x.n - p.Q + 1 + (first_row + r) / p.H : x.n; };
    const int see0 = sees(row0), see1 = sees(row0 + 8), least = x.n - p.Q + 1 + first_row / p.H;
    float m0 = kNegInf, m1 = kNegInf, l0 = 0.f, l1 = 0.f;
#pragma unroll 1
    for (int t = x.t0; t < x.t1; ++t, ++g) {
      const uint32_t st = g % G::NS;
      const int k0 = t * TK;
      wait_cap(&c.sfull[g & 1], (g >> 1) & 1, &c.abort, p.hdr);
      wait_cap(&c.full[st], (g / G::NS) & 1, &c.abort, p.hdr);   // (complete: for what its writers left in `dead`)
      __syncwarp();
      tc_fence_after();
      const uint32_t dead = *reinterpret_cast<const volatile uint32_t *>(&c.dead[st]);
      float s[NV];
      float x0 = kNegInf, x1 = kNegInf;
      if (act) {
        tmem_ld_16(tmem + lane_off + kColS + (g & 1) * TK, s);
#pragma unroll
        for (int i = 0; i < NV; ++i) s[i] *= f;
        if (k0 + TK > least || dead) {
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int key = (i >> 2) * 8 + 2 * qd + (i & 1);
            if (k0 + key >= ((i & 2) ? see1 : see0) || ((dead >> (key >> 4)) & 1)) s[i] = kNegInf;
          }
        }
#pragma unroll
        for (int i = 0; i < NV; i += 4) {
          x0 = fmaxf(x0, fmaxf(s[i], s[i + 1]));
          x1 = fmaxf(x1, fmaxf(s[i + 2], s[i + 3]));
        }
      }
      // ---- the running maximum moves when some score passes it by 2^kLazy
      bool waited = false;              // for the product before this one
      if (named_sync_or(kBarSoft, 128, act && (x0 > m0 + kLazy || x1 > m1 + kLazy))) {
        if (act) {
#pragma unroll
          for (int o = 1; o < 4; o <<= 1) {
            x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, o));
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, o));
          }
          x0 = fmaxf(x0, m0);
          x1 = fmaxf(x1, m1);
          const float a0 = x0 == kNegInf ? 1.f : ex2_approx(m0 - x0), a1 = x1 == kNegInf ? 1.f : ex2_approx(m1 - x1);
          m0 = x0;
          m1 = x1;
          l0 *= a0;
          l1 *= a1;
          if (qd == 0) {
            c.fac[row0] = a0;
            c.fac[row0 + 8] = a1;
          }
        }
        if (t > x.t0) {
          wait_cap(&c.odone[(g - 1) & 1], ((g - 1) >> 1) & 1, &c.abort, p.hdr);
          waited = true;
          named_sync(kBarSoft, 128);
          tc_fence_after();
#pragma unroll 1
          for (int ch = 0; ch < 4 * N; ch += 16) {
            float o[16];
            tmem_ld16(tmem + lane_off + kColO + ch, o);
            uint32_t v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(o[i] * c.fac[(ch + i) % N]);
            tmem_st16(tmem + lane_off + kColO + ch, v);
          }
          tmem_st_wait();
        }
      }
      // ---- weights
      if (act) {
        const float u0 = m0 == kNegInf ? 0.f : m0, u1 = m1 == kNegInf ? 0.f : m1;
#pragma unroll
        for (int i = 0; i < NV; i += 4) {
          s[i] = ex2_approx(s[i] - u0);
          s[i + 1] = ex2_approx(s[i + 1] - u0);
          s[i + 2] = ex2_approx(s[i + 2] - u1);
          s[i + 3] = ex2_approx(s[i + 3] - u1);
          l0 += s[i] + s[i + 1];
          l1 += s[i + 2] + s[i + 3];
        }
      }
      // the place of P is free once the product that read it last is complete
      if (!waited && g >= G::PB)
        wait_cap(&c.odone[(g - G::PB) & 1], ((g - G::PB) >> 1) & 1, &c.abort, p.hdr);
      if (act) {
        auto pack = [](float a, float b) { return FP8 ? tc::f2_to_h2(a, b) : tc::f2_to_bf2(a, b); };
        const uint32_t at = sP + row0 * 128 + 4 * qd;   // (row0 + 8 has the same place in its eight rows)
#pragma unroll
        for (int i = 0; i < TK / 8; ++i) {
          const uint32_t o = ((uint32_t)(i + (g % G::PB) * 4) ^ (row0 & 7)) << 4;
          sts_u32(at + o, pack(s[4 * i], s[4 * i + 1]));
          sts_u32(at + 1024 + o, pack(s[4 * i + 2], s[4 * i + 3]));
        }
      }
      // rows that no query sees may hold anything: zeros, for a zero weight times them must be zero
      if (k0 + TK > x.n || dead) {
        const uint32_t base = smem_u32(smem + G::OFF_K + st * G::STAGE);
        for (int i = tid; i < TK * 64; i += 128) {   // 16-byte pieces
          const int key = i >> 6;
          if (k0 + key >= x.n || ((dead >> (key >> 4)) & 1))
            sts_u4(base + (key >> 3) * 8192 + ((i >> 3) & 7) * 1024 + (key & 7) * 128 + (i & 7) * 16, 0, 0, 0, 0);
        }
      }
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.pready[g & 1]);
    }
    // ---- the sums, the last product, the output
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, o);
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
    const bool whole = x.whole();
    const long long slot = whole ? 0 : ((long long)(2 * worker + (x.first ? 0 : 1)) * p.S + sub) * p.R;
    named_sync(kBarSoft, 128);   // the factors of the last rescale have been read
    if (act && qd == 0) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = row0 + 8 * k;
        const float l = k ? l1 : l0, m = k ? m1 : m0;
        c.fac[r] = l != 0.f ? p.kv.g / l : 0.f;   // (0: the row saw no key; a NaN among its scores goes on)
        const float lse = l != 0.f ? (m + log2f(l)) * 0.69314718055994531f : kNegInf;
        if (r < rows) {
          if (!whole) p.part_lse[slot + r] = lse;
          else if (p.lse_out) p.lse_out[r_out + r] = lse;
        }
      }
    }
    wait_cap(&c.odone[(g - 1) & 1], ((g - 1) >> 1) & 1, &c.abort, p.hdr);
    named_sync(kBarSoft, 128);
    tc_fence_after();
    const bool wide = !whole || p.out_fp32;
    float *const of = whole ? static_cast<float *>(p.out) + r_out * kLatent : p.part_o + slot * kLatent;
    __nv_bfloat16 *const ob = static_cast<__nv_bfloat16 *>(p.out) + r_out * kLatent;
#pragma unroll 1
    for (int ch = 0; ch < 4 * N; ch += 16) {
      float o[16];
      tmem_ld16(tmem + lane_off + kColO + ch, o);
      const int d = ch / N * 128 + w * 32 + lane, r0 = ch % N;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (r0 + i >= rows) break;
        const float inv = c.fac[r0 + i], v = inv != 0.f ? o[i] * inv : 0.f;
        if (wide) of[(size_t)(r0 + i) * kLatent + d] = v;
        else ob[(size_t)(r0 + i) * kLatent + d] = __float2bfloat16_rn(v);
      }
    }
    tc_fence_before();
    named_sync(kBarSoft, 128);   // every warp has read O and the factors
  }
}

template <bool FP8, int N>
__global__ void __launch_bounds__(Geo<FP8, N>::THREADS, 1)
    latent_decode_kernel(const AbsorbedParams p, const __grid_constant__ CUtensorMap mq,
                         const __grid_constant__ CUtensorMap mc, const __grid_constant__ CUtensorMap mr) {
  using G = Geo<FP8, N>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  __shared__ Ctl c;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int worker = blockIdx.x / p.S, sub = blockIdx.x % p.S;
  griddep_launch();   // (only the join follows, which waits for this grid)
  if (warp == G::WARP_S) {
    tmem_alloc(&c.tmem, 512);
    tmem_relinquish();
  } else if (tid == 0) {
    for (int i = 0; i < G::NS; ++i) {
      mbar_init(&c.full[i], FP8 ? G::FWARPS : G::PG);
      mbar_init(&c.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.sfull[i], 1);
      mbar_init(&c.odone[i], 1);
      mbar_init(&c.pready[i], 4);
    }
    mbar_init(&c.qfull, FP8 ? G::QWARPS : 1);
    mbar_init(&c.qfree, 1);
    mbar_init(&c.done, 2);
    c.abort = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  find_run<G::TK>(p, c, worker, blockIdx.x == 0);
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, c.tmem, 0);
  if (warp < 4) {
    role_softmax<FP8, N>(p, smem, c, tmem, worker, sub);
  } else if (warp == G::WARP_S) {
    role_scores<FP8, N>(p, smem, c, tmem);
  } else if (warp == G::WARP_O) {
    role_output<FP8, N>(p, smem, c, tmem);
  } else if (warp < G::WARP_F) {
    role_query<FP8, N>(p, &mq, smem, c, sub, tid - G::WARP_Q * 32);
  } else if (warp < G::WARP_F + G::FWARPS) {
    if constexpr (FP8) role_dequant<N>(p, smem + G::OFF_K, c, tid - G::WARP_F * 32);
    else role_copy<N>(p, &mc, &mr, smem + G::OFF_K, c);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == G::WARP_S) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
    griddep_wait();   // the grid does not end before its header is cleared
  }
}

// ----------------------------------------------------------------- the join

// one CTA a row: zeros where there is no key, the joined pieces where a sequence's
// tiles went to several workers
__global__ void __launch_bounds__(128) latent_join_kernel(const AbsorbedParams p) {
  griddep_wait();   // the pieces are complete
  const int all = p.Q * p.H, row = blockIdx.x, b = row / all, r = row % all;
  const int tiles = p.starts[b + 1] - p.starts[b], tid = threadIdx.x;
  const int grp = r / p.R, sets = p.RG / p.S;
  long long slot0 = 0;
  int parts = 0;
  bool skip = false;      // of the first worker's slots
  if (tiles > 0) {
    const long long run = run_of(p, (long long)p.starts[p.B] * sets);
    const long long a = (long long)p.starts[b] * sets + (long long)(grp / p.S) * tiles;
    const int c0 = (int)(a / run), c1 = (int)((a + tiles - 1) / run);
    if (c0 == c1) return;   // written by the attention kernel
    parts = c1 - c0 + 1;
    slot0 = c0;
    skip = a != c0 * run;   // its piece is not the worker's first
  }
  auto at = [&](int k) {   // row of piece k among the partial ones
    return ((2 * (slot0 + k) + (k == 0 && skip ? 1 : 0)) * p.S + grp % p.S) * p.R + r % p.R;
  };
  float M = kNegInf;
  for (int k = 0; k < parts; ++k) M = fmaxf(M, p.part_lse[at(k)]);
  float sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = 0; k < parts; ++k) {
    const long long from = at(k);
    const float ls = p.part_lse[from];
    const float4 x = reinterpret_cast<const float4 *>(p.part_o + from * kLatent)[tid];
    if (ls == kNegInf) continue;
    const float wt = expf(ls - M);   // (a NaN among a piece's scores is in its lse)
    sum += wt;
    acc.x += wt * x.x;
    acc.y += wt * x.y;
    acc.z += wt * x.z;
    acc.w += wt * x.w;
  }
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  const size_t to = (size_t)row * kLatent + 4 * tid;
  if (p.out_fp32)
    *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + to) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  else
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + to) =
        make_uint2(tc::f2_to_bf2(acc.x * inv, acc.y * inv), tc::f2_to_bf2(acc.z * inv, acc.w * inv));
  if (tid == 0 && p.lse_out) p.lse_out[row] = sum != 0.f ? M + logf(sum) : kNegInf;
}

template <bool FP8, int N>
cudaError_t launch_n(const AbsorbedParams &p, const CUtensorMap &mc, const CUtensorMap &mr, cudaStream_t s) {
  using G = Geo<FP8, N>;
  CUtensorMap mq;
  std::memset(&mq, 0, sizeof mq);
  if (!FP8) {
    const uint64_t dims[2] = {(uint64_t)kRow, (uint64_t)p.B * p.Q * p.H}, strides[1] = {kRow * 2};
    const uint32_t box[2] = {64, (uint32_t)N};
    if (!make_map(&mq, p.q, 2, dims, strides, box)) return cudaErrorInvalidValue;
  }
  auto kern = latent_decode_kernel<FP8, N>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, (unsigned)(p.workers * p.S), G::THREADS, G::SMEM, s, p, mq, mc, mr);
}

template <bool FP8>
cudaError_t launch_fmt(const AbsorbedParams &p, const CUtensorMap &mc, const CUtensorMap &mr, cudaStream_t s) {
  if (p.R <= 16) return launch_n<FP8, 16>(p, mc, mr, s);
  if (p.R <= 32) return launch_n<FP8, 32>(p, mc, mr, s);
  return launch_n<FP8, 64>(p, mc, mr, s);
}

// CTAs at once: one per SM of this GPU (another count would only split the work worse)
constexpr int kSms = 152;

}  // namespace

DecodePlan plan_latent_decode(int B, int Q, int H, int max_seq_len) {
  DecodePlan d;
  const int rows = Q * H, groups = (rows + kMaxRows - 1) / kMaxRows;
  d.RG = groups <= 8 ? groups : (groups + 7) / 8 * 8;
  d.S = groups <= 8 ? groups : 8;
  d.R = (rows + d.RG - 1) / d.RG;
  const long long tiles = (long long)B * (d.RG / d.S) * ((max_seq_len + 31LL) / 32);
  const long long most = kSms / d.S;
  d.workers = (int)(tiles < 1 ? 1 : tiles < most ? tiles : most);
  return d;
}

cudaError_t launch_latent_decode(const AbsorbedParams &p, cudaStream_t s) {
  const bool fp8 = p.kv.dtype == PA_KV_FP8;
  CUtensorMap mc, mr;
  std::memset(&mc, 0, sizeof mc);
  std::memset(&mr, 0, sizeof mr);
  if (!fp8) {
    const uint64_t nb = (uint64_t)p.kv.num_blocks;
    const uint64_t dc[4] = {64, 8, 8, nb * 2}, sc[3] = {kLatent * 2, 128, 8 * kLatent * 2};
    const uint32_t bc[4] = {64, 8, 8, 2};
    const uint64_t dr[2] = {kRope, nb * kBlock}, sr[1] = {kRope * 2};
    const uint32_t br[2] = {kRope, kBlock};
    if (!make_map(&mc, p.kv.latent, 4, dc, sc, bc) || !make_map(&mr, p.kv.rope, 2, dr, sr, br))
      return cudaErrorInvalidValue;
  }
  cudaError_t e = fp8 ? launch_fmt<true>(p, mc, mr, s) : launch_fmt<false>(p, mc, mr, s);
  if (e != cudaSuccess) return e;
  return launch_pdl(latent_join_kernel, (unsigned)(p.B * p.Q * p.H), 128, 0, s, p);
}

}  // namespace lat
}  // namespace pa
